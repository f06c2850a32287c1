// Attention of chunks of new tokens over a paged cache: tiled S = Q K^T, online softmax and
// O += P V on the tensor cores, as in the contiguous forward (FlashAttention deep-read
// report, sections 2.4 and 3.2), with pages gathered tile by tile, ragged batches and query
// heads that share K/V heads.
//
// A query tile is 128 rows of one K/V head: TT = 128 / G tokens times the G = H / Hkv heads
// that read it (row r = t * G + g), so that K and V are read once for all of them. The list
// of (sequence, K/V head, query tile, 128-key tile) places is divided equally among the CTAs
// (one per SM) by the lengths found on the device: chunks of any lengths keep all SMs busy,
// and few query tiles over a long cache are split along the keys. A query tile that is cut
// leaves normalised pieces for the merge kernel.
//
// Roles of a CTA (the head-dimension-128 forward's shape, here for 64 too):
//   warps 0-3, 4-7  softmax warpgroups g = 0, 1: key tiles at even and odd positions of a
//                   piece (thread = query row), each with its own m, l, O in tensor memory;
//                   the epilogue merges the two
//   warps 8, 11     K and V tiles, one TMA box per page (or 16 .. 128 rows of it): into the K
//                   and V rings, or codes into staging rings (e4m3)
//   warps 9, 10     S issuer, which also loads Q, and PV issuer (one lane each)
//   warp 11         also works out the CTA's pieces, ahead of the others, who take them from a
//                   ring in shared memory (the divisions and loads behind a piece took each
//                   role 3000 cycles, half of what a piece of 4 key tiles takes)
//   warps 12-19     e4m3 only: turn staged codes, and Q, into f16 tiles with the rows' scales
//                   folded in; the products then run in f16, and P is f16 too
// Keys behind a sequence are masked by their number; V's rows there are made zero, since a
// weight of zero would not hide a NaN.
//
// Bounds: for chunks the tensor core (1024 cycles of products per 128 x 128 tile at d = 128, of
// 1500 measured with a bf16 cache; each warpgroup's chain of scores, maximum, exponentials and
// the handshakes with the products is the rest); with few rows HBM; from an e4m3 cache the
// conversion, which takes registers, issue slots and bandwidth of shared memory from the softmax,
// and the chain that goes from a PV product over the S that takes its place to the next P. us a
// tile and SM (8 K/V heads, 16 query tiles of 512 key tiles each): d = 128 bf16 0.83, e4m3 1.42
// (when it took 1.39, without the conversion 1.21, without the exponentials too 0.95); d = 64
// bf16 0.75, e4m3 1.05.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_paged_plan.cuh"

namespace fa {

namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kKWarp = 8;
constexpr int kSIssuer = 9;
constexpr int kPvIssuer = 10;
constexpr int kVWarp = 11;
constexpr int kConvWarp = 12;  // first of the converters (e4m3)
constexpr int kConvWarps = 8;

template <int D, bool E4M3>
struct ChunkL {
  static constexpr int kWarps = E4M3 ? kConvWarp + kConvWarps : 12;
  static constexpr int kThreads = kWarps * 32;
  // Registers per thread at launch, and as the warpgroups share them out afterwards.
  static constexpr int kRegsLaunch = E4M3 ? 96 : 168;
  // (e4m3, measured us per 128 x 128 tile and SM for softmax, aux, converters: d = 128 144, 64, 64
  // 1.47, 160, 64, 48 1.49, 128, 64, 80 1.50; d = 64 160, 64, 48 1.05, 144, 64, 64 1.25. These and
  // the comparisons below are from before later steps, which took 1.47 to 1.4.) At 96 registers the
  // e4m3 kernels spill: 368 bytes of stores and 404 of loads at d = 128, 100 and 136 at d = 64.
  static constexpr int kRegsSoftmax = E4M3 ? (D == 64 ? 160 : 144) : 216;
  static constexpr int kRegsAux = E4M3 ? 64 : 72;   // producers and issuers
  static constexpr int kRegsConv = E4M3 ? (D == 64 ? 48 : 64) : 0;  // converters
  static_assert(256 * kRegsSoftmax + 128 * kRegsAux + (kThreads - 384) * kRegsConv <=
                    kThreads * kRegsLaunch,
                "register reallocation exceeds the block's launch allocation");
  static constexpr int kTileBytes = kTile * D * 2;   // a 128 x D 16-bit tile
  // P_g: in shared memory (bf16), or in tensor memory (f16, e4m3): there the converters need the
  // room and the bandwidth of shared memory (us per tile with P in shared memory and in tensor
  // memory: e4m3 d = 128 1.71 and 1.47, d = 64 1.11 and 1.05).
  static constexpr int kPBytes = E4M3 ? 0 : kTile * kTile * 2;
  static constexpr int kChunks = D / 64;             // 64-column (128-byte) swizzle chunks
  // Ring depths; e4m3: of tiles ready for the products, and of staged codes (us per tile at d =
  // 128 with 2, 1, 3, 2 tiles of K, V, K's codes, V's codes 1.47; 2, 2, 2, 1 1.67; 1, 1, 4, 3
  // 1.49; 1, 2, 2, 3 1.50).
  static constexpr int kKStages = D == 64 && !E4M3 ? 4 : 2;
  static constexpr int kVStages = D == 128 && E4M3 ? 1 : kKStages;
  static constexpr int kCkStages = E4M3 ? (D == 64 ? 4 : 3) : 0;
  static constexpr int kCvStages = E4M3 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int kCodeBytes = kTile * D;
  static constexpr int kPieces = 4;                  // ring of pieces
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kPOff = kVOff + kVStages * kTileBytes;
  static constexpr int kCOff = kPOff + 2 * kPBytes;
  static constexpr int kCvOff = kCOff + kCkStages * kCodeBytes;
  static constexpr int kBarOff = kCvOff + kCvStages * kCodeBytes;
  // q_full, q_empty, q_ready, K and V rings (full, empty), their staging rings (full, empty),
  // piece ring (full, empty), s_full[2], s_free[2], p_full[2], pv_done[2], o_free, xbar[4],
  // v_tail, drain, drain2, stall
  static constexpr int kNumBars = 3 + 2 * (kKStages + kVStages) + 2 * (kCkStages + kCvStages) + 2 * kPieces + 8 + 1 + 4 + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;          // abort flag, TMEM address
  // e4m3: the scale bytes of staged tiles (K's stages: K's and V's; V's stages: V's); the
  // scales of the latest tiles and Q's row exponents of the latest pieces, for the softmax.
  // Tile n's slot is written when K's tile n is converted, so after the S product of tile n -
  // kKStages; that one waited until its warpgroup had read the tile before (S, and before it the
  // slot). The other warpgroup has then read all but its latest tile in front of it: where a
  // piece of an odd number of tiles ends, the next one begins with the same warpgroup, which
  // leaves tile n - kKStages - 2 unread, and none before that (a warpgroup enters a piece once
  // both have read all of the piece before). A piece's exponents are written after all S products
  // of the piece before, so when both warpgroups have left the piece before that one's
  // predecessor.
  static constexpr int kScaleSlots = E4M3 ? 8 : 0;
  static constexpr int kQExpSlots = E4M3 ? 4 : 0;
  static_assert(!E4M3 || kScaleSlots >= kKStages + 3, "a slot is rewritten before it is read");
  static constexpr int kPieceOff = (kMiscOff + 16 + 15) / 16 * 16;
  static constexpr int kBytesOff = kPieceOff + 48 * kPieces;
  static constexpr int kScaleOff = kBytesOff + kTile * (2 * kCkStages + kCvStages);
  static constexpr int kQExpOff = kScaleOff + 16 * kScaleSlots;
  static constexpr int kFactorOff = kQExpOff + kTile * kQExpSlots;  // f16 factors of K's and V's rows
  static constexpr int kXchOff = kFactorOff + (E4M3 ? 4 * kTile : 0);  // (m, l) per warpgroup and row
  // the plan's scratch is used before the exchange area is
  static constexpr int kPlanOff = kXchOff;
  static constexpr int kSmemBytes = kXchOff + 2 * kTile * 8;
  static_assert(kSmemBytes <= 232448, "shared memory exceeds the per-block limit");
  __device__ static constexpr uint32_t col_s(int g) { return 128u * static_cast<uint32_t>(g); }
  __device__ static constexpr uint32_t col_o(int g) { return 256u + 128u * static_cast<uint32_t>(g); }
  // e4m3: P_g's 64 columns, beside O_g where it leaves them, else in the second half of S_g
  __device__ static constexpr uint32_t col_p(int g) { return (D == 64 ? col_o(g) : col_s(g)) + 64u; }
  static constexpr bool kPInS = E4M3 && D == 128;
};

struct Bars {
  uint32_t q_full, q_empty, q_ready;
  BarRun k_full, k_empty, v_full, v_empty;      // ring stages
  BarRun ck_full, ck_empty, cv_full, cv_empty;  // staging rings (e4m3)
  BarRun pc_full, pc_empty;                     // pieces
  BarRun s_full, s_free, p_full, pv_done;   // per softmax warpgroup
  uint32_t o_free;
  BarRun xbar;
  uint32_t v_tail, drain, drain2, stall;
};

// Key tiles of a unit (query tile qt of a sequence): places n >= 1, of which the first nr
// are tiles jf, jf + 1, ... (a unit whose rows see no key has one place and no tile).
struct Tiles {
  int jf, nr, n;
};
__device__ __forceinline__ Tiles tiles_of(const PagedAttnArgs& a, const PagedSeq& s, int tt, int qt) {
  const int t_lo = qt * tt, t_hi = min(s.nq, t_lo + tt);
  const int pos = s.len - s.nq;
  const int hi = a.causal ? min(s.len, pos + t_hi) : s.len;  // keys [lo, hi) for some row
  const int lo = a.wl >= 0 ? max(0, pos + t_lo - a.wl) : 0;
  Tiles r;
  r.jf = lo / kTile;
  r.nr = hi > lo ? (hi + kTile - 1) / kTile - r.jf : 0;
  r.n = r.nr > 0 ? r.nr : 1;
  return r;
}

// A place in the list of units (sequence, K/V head, query tile).
struct Unit {
  int b, h, qt, n_qt;
  PagedSeq s;
  __device__ __forceinline__ void seq(const PagedAttnArgs& a) {
    s = paged_attn_seq(a.c, b);
    n_qt = (s.nq + a.tt - 1) / a.tt;
  }
  __device__ __forceinline__ void at(unsigned x) {  // its unit x
    h = static_cast<int>(x / static_cast<unsigned>(n_qt));
    qt = static_cast<int>(x) - h * n_qt;
  }
  // k units further on, by a warp whose lanes all hold the same unit.
  template <bool E4M3>
  __device__ __forceinline__ void advance(const PagedAttnArgs& a, int k);
};

// The units of 32 sequences, one a lane, and which they are in the list of all. Of use to a
// whole warp that looks for units further and further on: taking sequences one by one, each a
// load from L2, 1023 single tokens beside a chunk took 400 us of planning.
struct Window {
  int b0;
  unsigned from, all, inc;  // units before the window; in it; up to the lane's sequence
  PagedSeq s;
  int n_qt;
  // The window at sequence x, with `before` units in front of it.
  __device__ __forceinline__ void load(const PagedAttnArgs& a, int x, unsigned before) {
    const int lane = threadIdx.x & 31;
    b0 = x;
    from = before;
    s = PagedSeq{0, 0, 0};
    if (b0 + lane < a.c.B) s = paged_attn_seq(a.c, b0 + lane);
    n_qt = (s.nq + a.tt - 1) / a.tt;
    inc = static_cast<unsigned>(n_qt * a.c.Hkv);  // (the units of a batch fit an int)
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, inc, k);
      if (lane >= k) inc += y;
    }
    all = __shfl_sync(0xffffffffu, inc, 31);
  }
  // Unit x, which may differ from lane to lane, but for every lane lies behind the window's
  // first sequence; b = B past the end. Moves the window on as far as that takes.
  __device__ __forceinline__ Unit find(const PagedAttnArgs& a, unsigned x) {
    Unit u;
    u.b = a.c.B;
    u.h = u.qt = u.n_qt = 0;
    u.s = PagedSeq{0, 0, 0};
    while (true) {
      const bool here = x >= from && x - from < all;
      const unsigned y = x - from;
      int i = 0;  // sequences that end at or before it
#pragma unroll
      for (int k = 16; k > 0; k >>= 1)
        if (__shfl_sync(0xffffffffu, inc, i + k - 1) <= y) i += k;
      const int n = __shfl_sync(0xffffffffu, n_qt, i);
      const unsigned before = __shfl_sync(0xffffffffu, inc - static_cast<unsigned>(n_qt * a.c.Hkv), i);
      const PagedSeq z = {__shfl_sync(0xffffffffu, s.t0, i), __shfl_sync(0xffffffffu, s.nq, i),
                          __shfl_sync(0xffffffffu, s.len, i)};
      if (here) {
        u.b = b0 + i;
        u.n_qt = n;
        u.s = z;
        u.at(y - before);
      }
      if (__all_sync(0xffffffffu, here || x < from) || b0 + 32 >= a.c.B) return u;
      load(a, b0 + 32, from + all);
    }
  }
};

// (Two forms of one search, chosen by what the compiler makes of the whole kernel, whose softmax
// this warp shares registers and instruction cache with: chunks of 512 tokens over 5000 keys on
// average, with the window and with loads of its own: bf16 148 and 142 us, e4m3 232 and 249.)
template <bool E4M3>
__device__ __forceinline__ void Unit::advance(const PagedAttnArgs& a, int k) {
  if (b >= a.c.B) return;
  unsigned x = static_cast<unsigned>(h * n_qt + qt + k);
  if (x < static_cast<unsigned>(n_qt * a.c.Hkv)) {
    at(x);
  } else if constexpr (E4M3) {
    Window w;
    w.load(a, b, 0u);
    *this = w.find(a, x);
  } else {
    const int lane = threadIdx.x & 31;
    int b0 = b;
    bool found = false;
    b = a.c.B;
    h = qt = n_qt = 0;
    for (; b0 < a.c.B; b0 += 32) {
      unsigned n = 0;
      if (b0 + lane < a.c.B)
        n = static_cast<unsigned>((paged_attn_seq(a.c, b0 + lane).nq + a.tt - 1) / a.tt * a.c.Hkv);
      unsigned inc = n;
#pragma unroll
      for (int j = 1; j < 32; j <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, j);
        if (lane >= j) inc += y;
      }
      const unsigned all = __shfl_sync(0xffffffffu, inc, 31);
      int i = 0;  // sequences that end at or before x
#pragma unroll
      for (int k = 16; k > 0; k >>= 1)
        if (__shfl_sync(0xffffffffu, inc, i + k - 1) <= x) i += k;
      const unsigned before = __shfl_sync(0xffffffffu, inc - n, i);
      found = x < all;
      x -= found ? before : all;
      if (found) {
        b = b0 + i;
        break;
      }
    }
    if (found) {
      seq(a);
      at(x);
    }
  }
}

// A piece as the roles need it: key tiles [j0, j0 + nt) (nt < 0: no piece is left) of the query
// tile whose first token is tok0 of its sequence, token row row0 of q and o, position pos0.
struct Piece {
  int b, h, qt, nt;
  int j0, len, pos0, row0;
  int rows, from_start, ends;
};

// A CTA's work, piece by piece. First `rounds` whole units,
// gridDim.x apart in the list, so that neighbouring CTAs take neighbouring query tiles of a
// head at the same time and share its K/V tiles in L2; then a run of the places behind
// those, cut where it begins and ends. The run's first unit, if another CTA began it, comes
// last: where runs are shorter than a unit, all CTAs then begin at a head's first key and
// differ by one jump only, so that at any time they read a head at two places, not at as
// many as there are CTAs. (16 query tiles of 512 key tiles each over 8 heads: with runs in
// the list's order alone K and V, 268 MB, came from HBM once per query tile, at 7 TB/s.)
template <bool E4M3>
struct Walk {
  Unit u;
  int rounds;                        // whole units left
  bool in_round, in_run;
  int run_b, run_h, run_qt, run_at;  // where the run begins: run_at places into that unit
  int tail;                          // places of that unit kept for last
  long long left;                    // places of the run left
  // the current piece
  int j0, nt;                        // its key tiles: j0, j0 + 1, ..., nt of them
  bool from_start, ends;

  __device__ __forceinline__ int piece(const PagedAttnArgs& a, int at, long long most) {
    const Tiles t = tiles_of(a, u.s, a.tt, u.qt);
    const int take = most < t.n - at ? static_cast<int>(most) : t.n - at;
    j0 = t.jf + at;
    nt = max(0, min(j0 + take, t.jf + t.nr) - j0);
    from_start = at == 0;
    ends = at + take == t.n;
    return take;
  }
  __device__ __forceinline__ void to_run(const PagedAttnArgs& a) {
    u.b = run_b;
    u.h = run_h;
    u.qt = run_qt;
    u.seq(a);
  }
  // Next piece; false when there is none.
  __device__ __forceinline__ bool next(const PagedAttnArgs& a) {
    if (rounds > 0) {
      if (in_round) u.template advance<E4M3>(a, static_cast<int>(gridDim.x));
      in_round = true;
      --rounds;
      piece(a, 0, 0x7FFFFFFF);
      return true;
    }
    if (left > 0) {
      if (in_run) {
        u.template advance<E4M3>(a, 1);
      } else {
        in_run = true;
        to_run(a);
        if (run_at > 0) {
          tail = piece(a, run_at, left);
          left -= tail;
          if (left > 0) u.template advance<E4M3>(a, 1);
        }
      }
      if (left > 0) {
        left -= piece(a, 0, left);
        return true;
      }
    }
    if (tail > 0) {
      to_run(a);
      piece(a, run_at, tail);
      tail = 0;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// Arrives on an mbarrier once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Scores of keys outside [lo, hi) of a tile are masked.
template <int N>
__device__ __forceinline__ void mask_row(float* s, int lo, int hi) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k >= hi || k < lo) s[k] = -INFINITY;
}

// Maximum of N scores: three-input max over eight independent accumulators.
template <int N>
__device__ __forceinline__ float max_row(const float* s) {
  float mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = fmaxf(s[2 * k], s[2 * k + 1]);
#pragma unroll
  for (int k = 16; k < N; k += 16)
#pragma unroll
    for (int a = 0; a < 8; ++a) mx[a] = fmax3(mx[a], s[k + 2 * a], s[k + 2 * a + 1]);
  return fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

}  // namespace

template <int D, bool E4M3>
__global__ void __launch_bounds__(ChunkL<D, E4M3>::kThreads, 1)
    fa_paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const PagedAttnArgs args,
                          const int box_rows) {
  using L = ChunkL<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  PieceHeader* headers = static_cast<PieceHeader*>(args.headers);
  pdl_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) {
      record_error(args.sync.status, kStatusCuda);
      headers[blockIdx.x] = PieceHeader{-1, 0, 0, 1};
    }
    return;
  }
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff + 8);
  Bars bars;
  {
    int i = 0;
    auto nb = [&]() { return smem_u32(&bar_mem[i++]); };
    auto run = [&](int n) {
      const BarRun r{smem_u32(&bar_mem[i])};
      i += n;
      return r;
    };
    bars.q_full = nb();
    bars.q_empty = nb();
    bars.q_ready = nb();
    bars.k_full = run(L::kKStages);
    bars.k_empty = run(L::kKStages);
    bars.v_full = run(L::kVStages);
    bars.v_empty = run(L::kVStages);
    bars.ck_full = run(L::kCkStages);
    bars.ck_empty = run(L::kCkStages);
    bars.cv_full = run(L::kCvStages);
    bars.cv_empty = run(L::kCvStages);
    bars.pc_full = run(L::kPieces);
    bars.pc_empty = run(L::kPieces);
    bars.s_full = run(2);
    bars.s_free = run(2);
    bars.p_full = run(2);
    bars.pv_done = run(2);
    bars.o_free = nb();
    bars.xbar = run(4);
    bars.v_tail = nb();
    bars.drain = nb();
    bars.drain2 = nb();
    bars.stall = nb();
  }
  // (by a thread that has little to do for the plan, while the plan waits for its first loads)
  if (tid == kSIssuer * 32) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    *abort_flag = 0;
    mbar_init(bars.q_full, 1);
    mbar_init(bars.q_empty, 1);
    mbar_init(bars.q_ready, 4);
    // e4m3: K's or V's four converter warps arrive; bf16: the producer, with the bytes expected
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bars.k_full[s], E4M3 ? 4 : 1);
      mbar_init(bars.k_empty[s], 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(bars.v_full[s], E4M3 ? 4 : 1);
      mbar_init(bars.v_empty[s], 1);
    }
    // staged tiles: the producer's lane 0, and the lanes that copy scale bytes
    for (int s = 0; s < L::kCkStages; ++s) {
      mbar_init(bars.ck_full[s], 17);
      mbar_init(bars.ck_empty[s], 4);
    }
    for (int s = 0; s < L::kCvStages; ++s) {
      mbar_init(bars.cv_full[s], 9);
      mbar_init(bars.cv_empty[s], 4);
    }
    for (int s = 0; s < L::kPieces; ++s) {
      mbar_init(bars.pc_full[s], 1);
      // a lane of each softmax and converter warp, of the K producer and of the two issuers
      mbar_init(bars.pc_empty[s], kSoftmaxWarps + 3 + (E4M3 ? kConvWarps : 0));
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bars.s_full[g], 1);
      mbar_init(bars.s_free[g], 128);
      mbar_init(bars.p_full[g], 128);
      mbar_init(bars.pv_done[g], 1);
    }
    // o_free: the 256 softmax threads at the end of each epilogue, plus the PV issuer once
    // per piece after its own wait on the previous phase, so that no phase can complete
    // while the PV issuer still waits on the one before it
    mbar_init(bars.o_free, 257);
    for (int q = 0; q < 4; ++q) mbar_init(bars.xbar[q], 64);
    mbar_init(bars.v_tail, 1);
    mbar_init(bars.drain, 1);
    mbar_init(bars.drain2, 1);
    mbar_init(bars.stall, 1);
    fence_mbar_init();
  }
  // ---- this CTA's run of the list
  struct Plan {
    long long warp_sums[L::kWarps];
    long long rem, lo, hi;
    int b, h, qt, at;    // where the run begins
    int b0, h0, qt0;     // the first whole unit
    int last;
  };
  static_assert(sizeof(Plan) <= 2 * kTile * 8, "plan scratch");
  Plan* plan = reinterpret_cast<Plan*>(smem + L::kPlanOff);
  // Places of one K/V head of sequence b; long chunks are summed by the whole warp.
  int last = -1;  // the last sequence seen by this thread with several query tiles per head
  auto head_places = [&](int b) -> long long {
    PagedSeq s = {0, 0, 0};
    if (b < args.c.B) s = paged_attn_seq(args.c, b);
    const int n_qt = (s.nq + args.tt - 1) / args.tt;
    if (n_qt > 1) last = b;
    long long sum = 0;
    if (n_qt <= 2)
      for (int i = 0; i < n_qt; ++i) sum += tiles_of(args, s, args.tt, i).n;
    unsigned todo = __ballot_sync(0xffffffffu, n_qt > 2);
    while (todo != 0u) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      PagedSeq z;
      z.t0 = 0;
      z.nq = __shfl_sync(0xffffffffu, s.nq, src);
      z.len = __shfl_sync(0xffffffffu, s.len, src);
      const int n = (z.nq + args.tt - 1) / args.tt;
      long long part = 0;
      for (int i = lane; i < n; i += 32) part += tiles_of(args, z, args.tt, i).n;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) part += __shfl_xor_sync(0xffffffffu, part, k);
      if (lane == src) sum = part;
    }
    return sum;
  };
  long long total = 0, x0 = 0, at0 = 0, sum0 = 0;
  for (int b0 = 0; b0 < args.c.B; b0 += L::kThreads) {
    const long long x = head_places(b0 + tid) * args.c.Hkv;
    long long sum;
    const long long at = block_scan<L::kWarps>(x, plan->warp_sums, &sum);
    if (b0 == 0) {
      x0 = x;
      at0 = at;
      sum0 = sum;
    }
    total += sum;
  }
  if (tid == 0) plan->last = -1;
  __syncthreads();
  if (last >= 0) atomicMax(&plan->last, last);
  __syncthreads();
  last = plan->last;
  const int ctas = static_cast<int>(gridDim.x);
  const long long per = (total + ctas - 1) / ctas;
  // Whole units in rounds, as long as no CTA gets more than its share; thread c follows CTA
  // c. Behind the last sequence with several query tiles per head there is nothing to share,
  // and no round.
  long long load = 0;
  int rounds = 0;
  if (last >= 0) {
    Window w;
    Unit v;
    // (threads behind the last CTA's look up that one's units)
    unsigned x = static_cast<unsigned>(min(tid, ctas - 1));
    w.load(args, 0, 0u);
    v = w.find(args, x);
    if (tid == static_cast<int>(blockIdx.x) && v.b < args.c.B) {
      plan->b0 = v.b;
      plan->h0 = v.h;
      plan->qt0 = v.qt;
    }
    while (true) {
      const bool none = v.b >= args.c.B;
      const int n = none ? 0 : tiles_of(args, v.s, args.tt, v.qt).n;
      if (__syncthreads_or(none || load + n > per || (tid == 0 && v.b > last))) break;
      load += n;
      ++rounds;
      x += static_cast<unsigned>(ctas);
      v = w.find(args, x);
    }
  }
  // The places behind the rounds go to the CTAs in order, each up to its share. After rounds
  // that is one place more, so that no run is empty before the last: the pieces of a unit
  // then lie in consecutive CTAs.
  long long lo, hi;
  {
    const long long each = per + (rounds > 0 ? 1 : 0);
    long long loads;
    const long long before = block_scan<L::kWarps>(tid < ctas ? load : 0, plan->warp_sums, &loads);
    if (tid == static_cast<int>(blockIdx.x)) {
      const long long from = loads + tid * each - before;
      plan->lo = min(total, from);
      plan->hi = min(total, from + each - load);
    }
    __syncthreads();
    lo = plan->lo;
    hi = plan->hi;
  }
  if (lo >= hi && rounds == 0) {
    if (tid == 0) headers[blockIdx.x] = PieceHeader{-1, 0, 0, 1};
    return;
  }
  if (lo < hi) {
    long long base = 0;
    for (int b0 = 0; b0 < args.c.B && base <= lo; b0 += L::kThreads) {
      long long x = x0, sum = sum0, at = at0;
      if (b0 > 0) {
        x = head_places(b0 + tid) * args.c.Hkv;
        at = base + block_scan<L::kWarps>(x, plan->warp_sums, &sum);
      }
      if (at <= lo && lo < at + x) {
        const long long one = x / args.c.Hkv;  // places of one head
        plan->b = b0 + tid;
        plan->h = static_cast<int>((lo - at) / one);
        plan->rem = (lo - at) % one;
      }
      base += sum;
    }
  }
  __syncthreads();
  if (warp == 0 && lo < hi) {
    // the query tile within the head: 32 at a time
    const PagedSeq s = paged_attn_seq(args.c, plan->b);
    const int n_qt = (s.nq + args.tt - 1) / args.tt;
    long long rem = plan->rem;
    for (int i0 = 0; i0 < n_qt; i0 += 32) {
      const int n = i0 + lane < n_qt ? tiles_of(args, s, args.tt, i0 + lane).n : 0;
      long long inc = n;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += y;
      }
      if (inc - n <= rem && rem < inc) {
        plan->qt = i0 + lane;
        plan->at = static_cast<int>(rem - (inc - n));
      }
      const long long all = __shfl_sync(0xffffffffu, inc, 31);
      if (rem < all) break;
      rem -= all;
    }
  }

  if (warp == kSIssuer) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = args.sync.timeout_ns;
  Walk<E4M3> w;
  if (warp == kVWarp) {
    w.rounds = rounds;
    w.in_round = w.in_run = false;
    w.tail = 0;
    w.left = lo < hi ? hi - lo : 0;
    w.run_b = plan->b;
    w.run_h = plan->h;
    w.run_qt = plan->qt;
    w.run_at = plan->at;
    if (rounds > 0) {
      w.u.b = plan->b0;
      w.u.h = plan->h0;
      w.u.qt = plan->qt0;
      w.u.seq(args);
    }
  }
  __syncthreads();  // the plan has been read: its place is the exchange area from here on

  auto fail = [&](void) {
    *abort_flag = 1;
    record_error(args.sync.status, kStatusTimeout);
  };
  const uint32_t sQ = smem_u32(smem + L::kQOff);
  const uint32_t sK = smem_u32(smem + L::kKOff);
  const uint32_t sV = smem_u32(smem + L::kVOff);
  const uint32_t sP = smem_u32(smem + L::kPOff);

  // Piece n, from the ring; false if the wait for it ran out.
  const uint32_t sPc = smem_u32(smem + L::kPieceOff);
  auto read_piece = [&](int n) {
    const uint32_t at = sPc + (n % L::kPieces) * 48;
    const uint4 x = ld_shared_v4(at), y = ld_shared_v4(at + 16), z = ld_shared_v4(at + 32);
    Piece p;
    p.b = static_cast<int>(x.x);
    p.h = static_cast<int>(x.y);
    p.qt = static_cast<int>(x.z);
    p.nt = static_cast<int>(x.w);
    p.j0 = static_cast<int>(y.x);
    p.len = static_cast<int>(y.y);
    p.pos0 = static_cast<int>(y.z);
    p.row0 = static_cast<int>(y.w);
    p.rows = static_cast<int>(z.x);
    p.from_start = static_cast<int>(z.y);
    p.ends = static_cast<int>(z.z);
    return p;
  };
  auto wait_piece = [&](int n) {
    return mbar_wait_warp(bars.pc_full[n % L::kPieces], (n / L::kPieces) & 1, tmo, abort_flag);
  };
  auto wait_piece_lane = [&](int n) {
    return mbar_wait(bars.pc_full[n % L::kPieces], (n / L::kPieces) & 1, tmo, abort_flag);
  };
  auto leave_piece = [&](int n) {  // by one lane
    mbar_arrive(bars.pc_empty[n % L::kPieces]);
  };

  if (E4M3 && warp >= kConvWarp) {
    regs_dec<E4M3 ? L::kRegsConv : 24>();
    Piece pc = {};
    // ------------------------------------------------------------ converters
    // Four warps for K's tiles, four for V's (and for Q); warp x of them takes rows 32 x .. of
    // every tile: staged codes, as f16 into the tiles that the products read. A row's scale 2^E
    // is folded in relative to the tile's largest, 2^Et: code * 2^(E - Et) is exact in f16 down
    // to E - Et = -15, and off by at most 2^-25 below, 2^-33 of the largest value that the
    // tile's codes can stand for. The softmax
    // takes 2^Et into account. (Codes come by TMA, not by loads of these warps: a barrier
    // arrival waits for a thread's loads in flight, so none could be ahead.)
    // A pass covers 16 codes for each of 4 lanes of 8 rows, odd rows at the other half of the
    // row (d = 128), so that 8 lanes load, and store, on different banks.
    const bool is_k = warp < kConvWarp + 4;
    const int wx = (warp - kConvWarp) & 3;
    const int r0 = wx * 32;
    const int row8 = lane >> 2, u = lane & 3;
    const uint32_t c_ring = smem_u32(smem + (is_k ? L::kCOff : L::kCvOff));
    const uint32_t ring = is_k ? sK : sV;
    // scale bytes: of K and V in K's stages, of V in V's
    const uint32_t bytes = smem_u32(smem + L::kBytesOff) + (is_k ? 0 : 2 * kTile * L::kCkStages);
    const BarRun c_full = is_k ? bars.ck_full : bars.cv_full;
    const BarRun c_empty = is_k ? bars.ck_empty : bars.cv_empty;
    const BarRun full = is_k ? bars.k_full : bars.v_full;
    const BarRun empty = is_k ? bars.k_empty : bars.v_empty;
    const uint32_t c_stages = is_k ? L::kCkStages : L::kCvStages;
    uint32_t cs = 0, cph = 0, ts = 0, tph = 1, tile = 0, q_cnt = 0;
    bool ok = true;
    // The factors of the warp's rows, f16, for its conversion.
    const uint32_t sF = smem_u32(smem + L::kFactorOff) + (is_k ? 0 : 2 * kTile) + r0 * 2;
    // Et + 127 of a tile from the lane's four scale bytes (rows 4 lane ..). 127 if all of the
    // tile's rows are there with E of -14 .. 7, as those of a cache in use are: their factors
    // 2^E are normal in f16 as they stand. Else the largest, at least `least`, so that the
    // factors that the softmax makes of it stay normal.
    auto top_of = [&](uint32_t bytes, int j, int least) -> int {
      const int valid = pc.len - (j * kTile + lane * 4);
      const bool usual = valid >= 4 && __vcmpgeu4(bytes, 0x71717171u) == 0xFFFFFFFFu &&
                         __vcmpleu4(bytes, 0x86868686u) == 0xFFFFFFFFu;
      if (__all_sync(0xffffffffu, usual)) return 127;
      unsigned top = static_cast<unsigned>(least);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const unsigned e = (bytes >> (8 * k)) & 255u;
        if (k < valid && e != kScaleNaN) top = max(top, min(e, kScaleMax + 127u));
      }
      // 128 in place of 127, whose factors are those above
      const int t = static_cast<int>(__reduce_max_sync(0xffffffffu, top));
      return t == 127 ? 128 : t;
    };
    // Writes the factors 2^(E - Et) of the warp's rows: 0 for rows behind the sequence, a NaN
    // for rows marked so.
    auto write_factors = [&](uint32_t bytes, int j, int top) {
      if ((lane >> 3) == wx) {
        uint32_t f[2];
        if (top == 127) {  // bits (E + 15) << 10
          f[0] = (prmt(bytes, 0u, 0x4140u) - 0x00700070u) << 10;
          f[1] = (prmt(bytes, 0u, 0x4342u) - 0x00700070u) << 10;
        } else {
          const int valid = pc.len - (j * kTile + lane * 4);
          f[0] = f[1] = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = static_cast<int>((bytes >> (8 * k)) & 255u);
            const int x = min(e, kScaleMax + 127) - top;  // <= 0
            uint32_t h = x >= -14 ? static_cast<uint32_t>((x + 15) << 10)
                                  : (x >= -24 ? 1u << (x + 24) : 0u);
            if (e == kScaleNaN) h = 0x7E00u;
            if (k >= valid) h = 0u;
            f[k >> 1] |= h << (16 * (k & 1));
          }
        }
        st_shared_v2(sF + (lane & 7) * 8, f[0], f[1]);
      }
      __syncwarp();
    };
    auto convert_tile = [&](uint32_t dst, int j) {
      const int valid = pc.len - j * kTile;
      const uint32_t src = c_ring + cs * L::kCodeBytes;
#pragma unroll
      for (int rg = 0; rg < 4; ++rg) {
        const int row = r0 + rg * 8 + row8;
        const uint32_t fx = prmt(ld_shared_u16(sF + (rg * 8 + row8) * 2), 0u, 0x1010u);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          const int cc = L::kChunks == 2 ? (c ^ (row8 & 1)) : 0;
          uint4 y = ld_shared_v4(src + row * D + cc * 64 + u * 16);
          // a page may hold any code behind the sequence (7F times 0 would be a NaN)
          if (valid < kTile && row >= valid) y = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t line = dst + cc * 16384 + row * 128;
          uint32_t o[8];
          e4m3_to_f16(y.x, o[0], o[1]);
          e4m3_to_f16(y.y, o[2], o[3]);
          e4m3_to_f16(y.z, o[4], o[5]);
          e4m3_to_f16(y.w, o[6], o[7]);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = mul_f16x2(o[k], fx);
          st_shared_v4(line + (((2 * u) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          st_shared_v4(line + (((2 * u + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
      }
    };
    // The warp's rows of Q, bf16 -> f16 in place, each times 2^k that puts its
    // largest magnitude into [2^14, 2^15): f16 then holds all that bf16 held but for elements
    // below 2^-29 of it. (k is at most 60, which keeps the score's factor a normal number.)
    auto do_q = [&]() -> bool {
      if (!mbar_wait_warp(bars.q_full, q_cnt & 1, tmo, abort_flag)) return false;
      int8_t* q_exp = reinterpret_cast<int8_t*>(smem + L::kQExpOff) + (q_cnt & (L::kQExpSlots - 1u)) * kTile;
      const int r4 = lane >> 3, v = lane & 7;
#pragma unroll 1
      for (int pass = 0; pass < 8; ++pass) {
        const int row = r0 + pass * 4 + r4;
        const uint32_t at = sQ + row * 128 + ((v ^ (row & 7)) << 4);
        uint4 x[L::kChunks];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          x[c] = ld_shared_v4(at + c * 16384);
          constexpr uint32_t kAbs = 0x7FFF7FFFu;
          const uint32_t m = __vmaxu2(__vmaxu2(x[c].x & kAbs, x[c].y & kAbs),
                                      __vmaxu2(x[c].z & kAbs, x[c].w & kAbs));
          top = max(top, max(m & 0xFFFFu, m >> 16));
        }
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
        const int k2 = max(-114, min(60, 14 + 127 - static_cast<int>(top >> 7)));
        const float m = pow2i(k2);
        auto conv = [&](uint32_t y) {
          return pack_f16x2(__uint_as_float(y << 16) * m, __uint_as_float(y & 0xFFFF0000u) * m);
        };
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          st_shared_v4(at + c * 16384, conv(x[c].x), conv(x[c].y), conv(x[c].z), conv(x[c].w));
        if (v == 0) q_exp[row] = static_cast<int8_t>(k2);
      }
      ++q_cnt;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.q_ready);
      return true;
    };
    for (int n = 0;; ++n) {
      if (!wait_piece(n)) {
        ok = false;
        break;
      }
      pc = read_piece(n);
      if (pc.nt < 0) break;
      __syncwarp();
      if (lane == 0) leave_piece(n);
      if (!is_k && pc.nt > 0) ok = do_q();
      for (int i = 0; ok && i < pc.nt; ++i) {
        const int j = pc.j0 + i;
        if (!mbar_wait_warp(c_full[cs], cph, tmo, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t sb = bytes + cs * (is_k ? 2 * kTile : kTile) + lane * 4;
        const uint32_t mine = ld_shared_u32(sb);
        const int top = top_of(mine, j, is_k ? 127 - 40 : 127 - 60);
        write_factors(mine, j, top);
        // (the wait comes as late as it can: for V the last PV product, this and the next one
        // are a chain)
        if (!mbar_wait_warp(empty[ts], tph, tmo, abort_flag)) {
          ok = false;
          break;
        }
        convert_tile(ring + ts * L::kTileBytes, j);
        if (is_k && wx == 0) {
          const int ev = top_of(ld_shared_u32(sb + kTile), j, 127 - 60) - 127;  // V's, as V's warps find it
          if (lane == 0)
            reinterpret_cast<float4*>(smem + L::kScaleOff)[tile & (L::kScaleSlots - 1u)] =
                make_float4(pow2i(top - 127), static_cast<float>(ev), pow2i(-ev), 0.f);
          ++tile;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {  // the codes have been read, the tile is complete
          mbar_arrive(c_empty[cs]);
          mbar_arrive(full[ts]);
        }
        if (++cs == c_stages) {
          cs = 0;
          cph ^= 1u;
        }
        if (++ts == (is_k ? L::kKStages : L::kVStages)) {
          ts = 0;
          tph ^= 1u;
        }
      }
      if (!ok) break;
    }
    if (!ok) fail();
  } else if (warp >= kSoftmaxWarps) {
    regs_dec<L::kRegsAux>();
    Piece pc = {};
    const int n_box = kTile / box_rows;  // boxes of a key tile
    // Pages of 16-row groups, and the rows in them: lane l has group l % 8 of key tile j + l / 8,
    // so that one load serves four tiles. num_pages, which lies outside the maps and reads
    // as zeros, behind the sequence and for a page that is none.
    struct Rows {
      int page, slot;
    };
    auto rows_of = [&](int j) {
      // (unsigned: up to three tiles behind the sequence's last, which may lie beyond 31 bits)
      const unsigned at = static_cast<unsigned>(j + (lane >> 3)) * kTile + (lane & 7) * 16;
      Rows r;
      r.page = args.c.num_pages;
      r.slot = 0;
      if (at < static_cast<unsigned>(pc.len)) {
        const int pos = static_cast<int>(at);
        r.slot = page_row(args.c, pos);
        const int p = paged_page(args.c, pc.b, pos);
        if (p >= 0) r.page = p;
      }
      return r;
    };
    auto rows_at = [&](const Rows& r, int tile, int group) {
      const int from = (tile & 3) * 8 + (group & 7);
      Rows x;
      x.page = __shfl_sync(0xffffffffu, r.page, from);
      x.slot = __shfl_sync(0xffffffffu, r.slot, from);
      return x;
    };
    const int groups = box_rows / 16;
    if (warp == kKWarp || warp == kVWarp) {
      // ------------------------------------------------------------ producers
      // bf16: into the K or V ring. e4m3: codes into the staging ring, and the rows' scale
      // bytes, 16 of a page at a time: K's and V's with K's tile (the softmax needs what a
      // tile's scales come to before V is converted), V's again with V's.
      const bool is_k = warp == kKWarp;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      const BarRun full = E4M3 ? (is_k ? bars.ck_full : bars.cv_full) : (is_k ? bars.k_full : bars.v_full);
      const BarRun empty =
          E4M3 ? (is_k ? bars.ck_empty : bars.cv_empty) : (is_k ? bars.k_empty : bars.v_empty);
      const uint32_t ring = E4M3 ? smem_u32(smem + (is_k ? L::kCOff : L::kCvOff)) : (is_k ? sK : sV);
      constexpr int kBytes = E4M3 ? L::kCodeBytes : L::kTileBytes;
      const uint32_t stages =
          E4M3 ? (is_k ? L::kCkStages : L::kCvStages) : (is_k ? L::kKStages : L::kVStages);
      const uint32_t scale_ring = smem_u32(smem + L::kBytesOff) + (is_k ? 0 : 2 * kTile * L::kCkStages);
      const uint8_t* scales = is_k && lane < 8 ? args.c.k_scale : args.c.v_scale;
      const int scale_lanes = is_k ? 16 : 8;
      uint32_t it = 0, s = 0, ph = 1, tails = 0;
      bool ok = true;
      Piece ahead = {};
      for (int n = is_k ? 0 : -1; ok; ++n) {
        if (is_k) {
          if (!wait_piece(n)) {
            fail();
            ok = false;
            break;
          }
          pc = read_piece(n);
          __syncwarp();
          if (pc.nt >= 0 && lane == 0) leave_piece(n);
        } else {
          // this warp works out the pieces: the next one before it loads V of this one
          pc = ahead;
          if (n < 0 || pc.nt >= 0) {
            ahead.nt = -1;
            if (w.next(args)) {
              const int tok0 = w.u.qt * args.tt;
              ahead.b = w.u.b;
              ahead.h = w.u.h;
              ahead.qt = w.u.qt;
              ahead.nt = w.nt;
              ahead.j0 = w.j0;
              ahead.len = w.u.s.len;
              ahead.pos0 = w.u.s.len - w.u.s.nq + tok0;
              ahead.row0 = w.u.s.t0 + tok0;
              ahead.rows = min(w.u.s.nq - tok0, args.tt) * args.G;
              ahead.from_start = w.from_start;
              ahead.ends = w.ends;
            }
            const int x = (n + 1) % L::kPieces;
            if (!mbar_wait_warp(bars.pc_empty[x], (((n + 1) / L::kPieces) & 1) ^ 1, tmo, abort_flag)) {
              fail();
              ok = false;
              break;
            }
            if (lane == 0) {
              const uint32_t at = sPc + x * 48;
              st_shared_v4(at, ahead.b, ahead.h, ahead.qt, ahead.nt);
              st_shared_v4(at + 16, ahead.j0, ahead.len, ahead.pos0, ahead.row0);
              st_shared_v4(at + 32, ahead.rows, ahead.from_start, ahead.ends, 0);
              mbar_arrive(bars.pc_full[x]);
            }
            __syncwarp();
            if (n < 0) continue;
          }
        }
        if (pc.nt < 0) break;
        Rows rows = {0, 0};
        for (int i = 0; i < pc.nt; ++i) {
          const int j = pc.j0 + i;
          if ((i & 3) == 0) rows = rows_of(j);
          const Rows box = rows_at(rows, i, lane * groups);
          long long at = 0;
          bool there = false;
          if constexpr (E4M3) {
            const Rows row = rows_at(rows, i, lane);
            there = row.page < args.c.num_pages;  // if not, zeros
            if (there)
              at = (static_cast<long long>(row.page) * args.c.Hkv + pc.h) * args.c.page_size + row.slot;
          }
          if (!mbar_wait_warp(empty[s], ph, tmo, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t dst = ring + s * kBytes;
          const int valid = pc.len - j * kTile;
          // V's last tile: rows of its last page behind the sequence may hold anything, so it
          // comes on a barrier of its own and is handed on once they have been cleared
          const bool tail = !E4M3 && !is_k && valid < kTile;
          const uint32_t bar = tail ? bars.v_tail : full[s];
          if constexpr (E4M3) {
            if (lane < scale_lanes) {
              cp_async16(scale_ring + s * scale_lanes * 16 + lane * 16, scales + at, there);
              cp_async_arrive(bar);
            }
          }
          if (lane == 0) mbar_expect_tx(bar, kBytes);
          __syncwarp();
          if (lane < n_box) {
            if constexpr (E4M3) {
              tma_load_4d(dst + lane * box_rows * D, tm, 0, box.slot, pc.h, box.page, bar);
            } else {
              for (int c = 0; c < L::kChunks; ++c)
                tma_load_4d(dst + c * 16384 + lane * box_rows * 128, tm, c * 64, box.slot, pc.h,
                            box.page, bar);
            }
          }
          __syncwarp();
          if (tail) {
            ++tails;
            if (!mbar_wait_warp(bars.v_tail, (tails - 1) & 1, tmo, abort_flag)) {
              fail();  // the drain below waits for the load
              ok = false;
              break;
            }
            const int end = (valid + box_rows - 1) / box_rows * box_rows;
            for (int x = valid * 8 + lane; x < end * 8; x += 32)
              for (int c = 0; c < L::kChunks; ++c)
                st_shared_v4(dst + c * 16384 + x * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full[s]);
          }
          ++it;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // Drain: every load this warp issued must land before the CTA exits. Stage x was armed
      // for ring positions x, x + stages, ...; wait for the last one.
      if (tails > 0) mbar_wait_warp(bars.v_tail, (tails - 1) & 1, tmo, nullptr);
      for (uint32_t x = 0; x < stages; ++x)
        if (it > x) mbar_wait_warp(full[x], ((it - 1 - x) / stages) & 1, tmo, nullptr);
    } else if (warp == kSIssuer) {
      // ------------------------------------------------------------ S issuer
      if (lane == 0) {
        // S = Q K^T, both K-major; bf16, or f16 for a quantised cache
        constexpr uint32_t kIdS = E4M3 ? idesc_f16_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint64_t kStep = static_cast<uint64_t>(L::kTileBytes >> 4);
        const uint64_t dQ = sdesc_sw128(sQ, 16, 1024);
        const uint64_t dK0 = sdesc_sw128(sK, 16, 1024);
        const uint32_t q_bytes = static_cast<uint32_t>(L::kChunks * args.G * args.tt * 128);
        uint32_t s = 0, ph = 0, sf0 = 0, sf1 = 0;
        uint32_t q_cnt = 0;  // pieces with key tiles so far: those that have loaded Q
        bool seen0 = false, seen1 = false;
        bool ok = true;
        // Test hook: this barrier is never completed, so the bounded wait runs out.
        if (args.sync.inject_stall && !mbar_wait(bars.stall, 0, tmo, abort_flag)) {
          fail();
          ok = false;
        }
        for (int n = 0; ok; ++n) {
          if (!wait_piece_lane(n)) {
            fail();
            break;
          }
          pc = read_piece(n);
          if (pc.nt < 0) break;
          leave_piece(n);
          if (pc.nt > 0) {
            // Q is replaced once the last piece's S products have completed
            if (q_cnt > 0 && !mbar_wait(bars.q_empty, (q_cnt - 1) & 1, tmo, abort_flag)) {
              fail();
              break;
            }
            mbar_expect_tx(bars.q_full, q_bytes);
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(sQ + c * 16384, &tm_q, c * 64, pc.h * args.G, pc.row0,
                          bars.q_full);
            ++q_cnt;
            if (!mbar_wait(E4M3 ? bars.q_ready : bars.q_full, (q_cnt - 1) & 1, tmo, abort_flag)) {
              fail();
              break;
            }
          }
          for (int p = 0; p < pc.nt; ++p) {
            const int g = p & 1;
            if (!mbar_wait(bars.k_full[s], ph, tmo, abort_flag)) {
              ok = false;
              break;
            }
            // S_g is free once its warpgroup has read the previous S_g, or, with P_g in it, once
            // the previous PV_g has run.
            const BarRun s_free = L::kPInS ? bars.pv_done : bars.s_free;
            if (g == 0) {
              if (seen0 && !mbar_wait(s_free[0], sf0++ & 1, tmo, abort_flag)) {
                ok = false;
                break;
              }
              seen0 = true;
            } else {
              if (seen1 && !mbar_wait(s_free[1], sf1++ & 1, tmo, abort_flag)) {
                ok = false;
                break;
              }
              seen1 = true;
            }
            tc_fence_after();
            const uint64_t dk = dK0 + static_cast<uint64_t>(s) * kStep;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_ss(tmem + L::col_s(g), dQ + off, dk + off, kIdS, kk > 0 ? 1u : 0u);
            }
            mma_commit(bars.s_full[g]);
            mma_commit(bars.k_empty[s]);
            if (++s == L::kKStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) {
            fail();
            break;
          }
          if (pc.nt > 0) mma_commit(bars.q_empty);
        }
        if (q_cnt > 0) mbar_wait(bars.q_full, (q_cnt - 1) & 1, tmo, nullptr);
        // Drain: all issued MMAs must finish before tensor memory is released.
        mma_commit(bars.drain);
        mbar_wait(bars.drain, 0, tmo, nullptr);
      }
      __syncwarp();
    } else if (warp == kPvIssuer) {
      // ------------------------------------------------------------ PV issuer
      if (lane == 0) {
        // P K-major, V MN-major
        constexpr uint32_t kIdPV = E4M3 ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
        constexpr uint64_t kStep = static_cast<uint64_t>(L::kTileBytes >> 4);
        constexpr uint64_t kPStep = static_cast<uint64_t>(L::kPBytes >> 4);
        const uint64_t dP0 = sdesc_sw128(sP, 16, 1024);
        const uint64_t dV0 = sdesc_sw128(sV, 16384, 1024);
        uint32_t s = 0, ph = 0, pc0 = 0, pc1 = 0;
        bool ok = true;
        for (int count = 0; ok; ++count) {  // piece
          if (!wait_piece_lane(count)) {
            fail();
            break;
          }
          pc = read_piece(count);
          if (pc.nt < 0) break;
          leave_piece(count);
          // The first PV of a piece overwrites O_0 or O_1, which the previous piece's
          // epilogue reads: it waits for that epilogue (o_free).
          bool first_any = true, first0 = true, first1 = true;
          for (int p = 0; p < pc.nt; ++p) {
            const int g = p & 1;
            const uint32_t pc = g ? pc1 : pc0;
            if (!mbar_wait(bars.v_full[s], ph, tmo, abort_flag) ||
                !mbar_wait(bars.p_full[g], pc & 1, tmo, abort_flag)) {
              ok = false;
              break;
            }
            if (g) ++pc1; else ++pc0;
            if (first_any) {
              if (count > 0 && !mbar_wait(bars.o_free, (count - 1) & 1, tmo, abort_flag)) {
                ok = false;
                break;
              }
              mbar_arrive(bars.o_free);
              first_any = false;
            }
            tc_fence_after();
            const bool first = g ? first1 : first0;
            const uint64_t dp = dP0 + static_cast<uint64_t>(g) * kPStep;
            const uint64_t dv = dV0 + static_cast<uint64_t>(s) * kStep;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              const uint64_t v_at = dv + static_cast<uint64_t>((kk * 2048) >> 4);
              const uint32_t acc = (first && kk == 0) ? 0u : 1u;
              if constexpr (E4M3)
                mma_ts(tmem + L::col_o(g), tmem + L::col_p(g) + 8 * kk, v_at, kIdPV, acc);
              else
                mma_ss(tmem + L::col_o(g), dp + off, v_at, kIdPV, acc);
            }
            if (g) first1 = false; else first0 = false;
            mma_commit(bars.pv_done[g]);
            mma_commit(bars.v_empty[s]);
            if (++s == L::kVStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          // A piece without any PV still consumes the previous epilogue's handshake and
          // adds its own arrival.
          if (ok && first_any) {
            if (count > 0 && !mbar_wait(bars.o_free, (count - 1) & 1, tmo, abort_flag))
              ok = false;
            else
              mbar_arrive(bars.o_free);
          }
          if (!ok) {
            fail();
            break;
          }
        }
        mma_commit(bars.drain2);
        mbar_wait(bars.drain2, 0, tmo, nullptr);
      }
      __syncwarp();
    }
  } else {
    regs_inc<L::kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2;                 // warpgroup: key tiles at positions p, p % 2 == g
    const int quad = warp & 3;               // tensor-memory lane quadrant of this warp
    const int t = quad * 32 + lane;          // row within the query tile
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_base + L::col_s(g);
    const uint32_t tO = tmem + lane_base + L::col_o(g);
    const uint32_t tP = tmem + lane_base + L::col_p(g);  // e4m3
    // r / G for r < 128, G <= 128: the excess r / 65536 of the product stays below 1 / G
    auto token_of = [&](int r) {
      return static_cast<int>((static_cast<uint32_t>(r) * args.g_magic) >> 16);
    };
    // This row of P_g, with the row's swizzle phase (t mod 8) in address bits 4-6:
    // 16-byte unit v of the row then sits at prow ^ (v << 4).
    const uint32_t prow = sP + static_cast<uint32_t>(g * L::kPBytes + t * 128 + ((t & 7) << 4));
    float2* xch = reinterpret_cast<float2*>(smem + L::kXchOff);
    const float c_log2 = args.scale_log2;
    // e4m3: the tiles' scales and the row exponents of Q, as the converters leave them
    const float4* tile_scale = reinterpret_cast<const float4*>(smem + L::kScaleOff);
    const int8_t* q_exp = reinterpret_cast<const int8_t*>(smem + L::kQExpOff);
    uint32_t tile_cnt = 0, q_cnt = 0;  // key tiles, and pieces with any, before this piece
    float c_row = 0.f;
    uint32_t s_cnt = 0, pv_cnt = 0;
    bool ok = true;
    int count = 0;
    PieceHeader* left = &headers[blockIdx.x];
    if (tid == 0) *left = PieceHeader{-1, 0, 0, 1};
    while (true) {
      if (!wait_piece(count)) {
        fail();
        ok = false;
        break;
      }
      int nt, j0;
      // keys [key_lo, key_hi) are visible to this row
      int key_lo = 0, key_hi;
      {
        const Piece pc = read_piece(count);
        nt = pc.nt;
        j0 = pc.j0;
        key_hi = pc.len;
        const int pos = pc.pos0 + token_of(t);
        if (args.causal && pos + 1 < key_hi) key_hi = pos + 1;
        if (args.wl >= 0) key_lo = pos - args.wl;
      }
      if (nt < 0) break;
      float m_ref = -INFINITY;  // reference maximum, scaled log2 units
      float l_sum = 0.f;        // running sum of exp2(s*c - m_ref)
      int n_done = 0;           // key tiles of this warpgroup
      for (int p = g; p < nt; p += 2) {
        const int k0 = (j0 + p) * kTile;
        if (!mbar_wait_warp(bars.s_full[g], s_cnt & 1, tmo, abort_flag)) {
          fail();
          ok = false;
          break;
        }
        ++s_cnt;
        tc_fence_after();
        // A score's exponent is s * c_t + ev (log2 units): for a quantised cache with the scales
        // that Q's row and K's tile were given, and V's tile's scale 2^ev, which P carries so
        // that all tiles add to one O; l takes it out again.
        float c_t = c_log2, ev = 0.f, ev_inv = 1.f;
        if constexpr (E4M3) {
          if (n_done == 0)
            c_row = c_log2 * pow2i(-static_cast<int>(q_exp[(q_cnt & (L::kQExpSlots - 1u)) * kTile + t]));
          const float4 z = tile_scale[(tile_cnt + p) & (L::kScaleSlots - 1u)];
          c_t = c_row * z.x;
          ev = z.y;
          ev_inv = z.z;
        }
        // bf16: the whole row in registers at once. e4m3, where the converters need registers
        // and instruction cache: half a row at a time, in one loop.
        constexpr int kCols = E4M3 ? 64 : 128;
        float s[kCols];
        const bool edge = k0 < key_lo || k0 + kTile > key_hi;
        auto load_scores = [&](int c0) {
          uint32_t sr[kCols];
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tS + c0 + c * 32, &sr[c * 32]);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < kCols; ++k) s[k] = __uint_as_float(sr[k]);
        };
        auto release_scores = [&]() {  // the next S of this warpgroup may be written over it
          tc_fence_before();
          mbar_arrive(bars.s_free[g]);
        };
        bool grow = false;
        float alpha = 1.f;
        uint64_t nm2 = 0;  // what a score's exponent adds, twice
        // Takes the largest score of a row into the reference maximum, which moves when it would
        // be exceeded by more than 2^kRescale.
        auto refer_to = [&](float mx) {
          const float m_new = fmaxf(m_ref, E4M3 ? fmaf(mx, c_t, ev - kF16Lift) : mx * c_t);
          grow = m_new > m_ref + kRescale;
          if (grow) {
            alpha = ex2_approx(m_ref - m_new);  // 0 when m_ref = -inf
            l_sum *= alpha;
            m_ref = m_new;
          }
          const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
          const float nm = E4M3 ? ev - m_use : -m_use;
          nm2 = f2_pack(nm, nm);
        };
        const uint64_t c2 = f2_pack(c_t, c_t);
        uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};  // four packed partial sums
        constexpr int kPk = kCols / 2;
        uint32_t pk[kPk];
        bool pv_ok = true;
        // 128-byte swizzle: 16-byte unit v of the row's 64-key half h at v ^ (t & 7)
        auto store_half = [&](int h) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const int x = h * 32 + 4 * v;
            st_shared_v4((prow ^ static_cast<uint32_t>(v << 4)) + static_cast<uint32_t>(h * 16384),
                         pk[x], pk[x + 1], pk[x + 2], pk[x + 3]);
          }
        };
        auto wait_pv = [&]() -> bool {  // the previous PV, which reads P_g, has completed
          if (!mbar_wait_warp(bars.pv_done[g], pv_cnt & 1, tmo, abort_flag)) return false;
          ++pv_cnt;
          tc_fence_after();
          return true;
        };
        // P = 2^(s * c_t + nm) of N scores, rounded to bf16 for the product (at most 2^-8 of each
        // weight: its operands have one type, which is V's; a second product for what the rounding
        // leaves would cost half as many again as there are), or to f16 (2^-11, or 2^-32 of the
        // largest where that is more); l keeps fp32.
        auto weights = [&](const float* x, uint32_t* to) {
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float y0, y1;
            f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), c2, nm2), y0, y1);
            const float p0 = ex2_approx(y0);
            const float p1 = ex2_approx(y1);
            rs2[(e >> 1) & 3] = f2_add(rs2[(e >> 1) & 3], f2_pack(p0, p1));
            to[e >> 1] = E4M3 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
        };
        if constexpr (E4M3) {
          // The halves are loaded as 0, 1 (for the maximum; then 1's weights) and 0 again: P_g,
          // where it lies in S_g, takes the columns of half 1.
          float mx = -INFINITY;
#pragma unroll 1
          for (int step = 0; step < 3; ++step) {
            const int half = step & 1;
            load_scores(half * 64);
            if (step == 2 && !L::kPInS) release_scores();
            if (edge) mask_row<kCols>(s, key_lo - k0 - half * 64, key_hi - k0 - half * 64);
            if (step < 2) mx = fmaxf(mx, max_row<kCols>(s));
            if (step == 0) continue;
            if (step == 1) {
              refer_to(mx);
              if (n_done > 0 && !wait_pv()) {
                pv_ok = false;
                break;
              }
            }
            weights(s, pk);
            tmem_st32(tP + half * 32, pk);
          }
          tmem_st_wait();
        } else {
          load_scores(0);
          release_scores();
          if (edge) mask_row<kCols>(s, key_lo - k0, key_hi - k0);
          refer_to(max_row<kCols>(s));
          weights(s, pk);
          // The first half goes out now if the previous PV has already completed; otherwise the
          // second half's exponentials come first.
          const bool ready =
              n_done == 0 ||
              __all_sync(0xffffffffu, mbar_test_wait(bars.pv_done[g], pv_cnt & 1));
          if (ready) {
            if (n_done > 0) {
              ++pv_cnt;
              tc_fence_after();
            }
            store_half(0);
          }
          weights(s + kCols / 2, pk + kPk / 2);
          if (!ready) {
            pv_ok = wait_pv();
            if (pv_ok) store_half(0);
          }
          if (pv_ok) store_half(1);
        }
        if (!pv_ok) {
          fail();
          ok = false;
          break;
        }
        {
          const uint64_t t2 = f2_add(f2_add(rs2[0], rs2[1]), f2_add(rs2[2], rs2[3]));
          float r0, r1;
          f2_unpack(t2, r0, r1);
          l_sum += E4M3 ? (r0 + r1) * ev_inv : r0 + r1;
        }
        // Rescale the O_g row in tensor memory (the previous PV has completed).
        if (n_done > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
          tmem_st_wait();
        }
        // P_g's generic-proxy stores become visible to the tensor core's reads.
        if constexpr (!E4M3) fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bars.p_full[g]);
        ++n_done;
      }
      if (!ok) break;
      // ---- epilogue: merge the two warpgroups' partial softmaxes.
      // This warpgroup's last PV has completed once its pv_done phase has.
      if (n_done > 0) {
        if (!mbar_wait_warp(bars.pv_done[g], pv_cnt & 1, tmo, abort_flag)) {
          fail();
          ok = false;
          break;
        }
        ++pv_cnt;
      }
      // The exchange slots are reused once both warpgroups have finished the previous
      // piece's epilogue (o_free completes after every read of them).
      if (count > 0 && !mbar_wait_warp(bars.o_free, (count - 1) & 1, tmo, abort_flag)) {
        fail();
        ok = false;
        break;
      }
      xch[g * kTile + t] = make_float2(m_ref, l_sum);
      // The partner row (same lane quadrant, other warpgroup) arrives after its own last PV
      // has completed, so both O_0 and O_1 are final past this wait.
      mbar_arrive(bars.xbar[quad]);
      if (!mbar_wait_warp(bars.xbar[quad], count & 1, tmo, abort_flag)) {
        fail();
        ok = false;
        break;
      }
      tc_fence_after();
      const float2 other = xch[(1 - g) * kTile + t];
      const float m0 = g ? other.x : m_ref, l0 = g ? other.y : l_sum;
      const float m1 = g ? m_ref : other.x, l1 = g ? l_sum : other.y;
      const bool has0 = nt > 0, has1 = nt > 1;  // O_g was written
      const float m = fmaxf(m0, m1);
      // l is 0 where no key was seen, and a NaN stays one
      const float a0 = (l0 == 0.f) ? 0.f : ex2_approx(m0 - m);
      const float a1 = (l1 == 0.f) ? 0.f : ex2_approx(m1 - m);
      const float l = a0 * l0 + a1 * l1;
      const float inv = (l == 0.f) ? 0.f : 1.f / l;
      const float w0 = a0 * inv, w1 = a1 * inv;
      const float lse2 = (l == 0.f) ? -INFINITY : m + __log2f(l);  // log2 units
      const Piece pc = read_piece(count);
      const int head = pc.h * args.G;  // the tile's first query head
      const bool direct = pc.from_start && pc.ends;
      // This warpgroup writes output columns [D/2 g, D/2 g + D/2) from both O_0 and O_1.
      constexpr int kHalf = D / 2;
      if (direct && E4M3) {
        // P_g takes no shared memory here that rows could be gathered in: 32 bytes of a row, a
        // whole sector, at a time
        const int tk = token_of(t);
        const long long at = static_cast<long long>(pc.row0 + tk) * args.H + head + (t - tk * args.G);
#pragma unroll 1
        for (int c = 0; c < kHalf / 16; ++c) {
          const uint32_t col = static_cast<uint32_t>(kHalf * g + 16 * c);
          uint32_t o0[16], o1[16];
          if (has0) tmem_ld16(tmem + lane_base + L::col_o(0) + col, o0);
          if (has1) tmem_ld16(tmem + lane_base + L::col_o(1) + col, o1);
          tmem_ld_wait();
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v0 = 0.f, v1 = 0.f;
            if (has0) {
              v0 = __uint_as_float(o0[2 * k]) * w0;
              v1 = __uint_as_float(o0[2 * k + 1]) * w0;
            }
            if (has1) {
              v0 = fmaf(__uint_as_float(o1[2 * k]), w1, v0);
              v1 = fmaf(__uint_as_float(o1[2 * k + 1]), w1, v1);
            }
            pk[k] = pack_bf16x2(v0, v1);
          }
          if (t < pc.rows) {
            uint4* dst = reinterpret_cast<uint4*>(args.o + at * D + col);
            dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          }
        }
        if (t < pc.rows && g == 0) args.lse[at] = lse2 * kLn2;
      } else if (direct) {
        // Each warp first puts its 32 rows x D bytes into shared memory (rows of P_g that it
        // itself writes, free once its last PV has completed), then stores them so that
        // neighbouring lanes cover whole rows.
        constexpr int kUnits = kHalf / 8;  // 16-byte units of a row's half
        const uint32_t stage = sP + static_cast<uint32_t>(g * L::kPBytes + quad * 4096);
        const uint32_t srow = stage + static_cast<uint32_t>(lane * kHalf * 2);
#pragma unroll
        for (int c = 0; c < kHalf / 16; ++c) {  // 16 columns at a time (fewer live registers)
          const uint32_t col = static_cast<uint32_t>(kHalf * g + 16 * c);
          uint32_t o0[16], o1[16];
          if (has0) tmem_ld16(tmem + lane_base + L::col_o(0) + col, o0);
          if (has1) tmem_ld16(tmem + lane_base + L::col_o(1) + col, o1);
          tmem_ld_wait();
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v0 = 0.f, v1 = 0.f;
            if (has0) {
              v0 = __uint_as_float(o0[2 * k]) * w0;
              v1 = __uint_as_float(o0[2 * k + 1]) * w0;
            }
            if (has1) {
              v0 = fmaf(__uint_as_float(o1[2 * k]), w1, v0);
              v1 = fmaf(__uint_as_float(o1[2 * k + 1]), w1, v1);
            }
            pk[k] = pack_bf16x2(v0, v1);
          }
          const uint32_t z = static_cast<uint32_t>(lane & (kUnits - 1));
          st_shared_v4(srow + (((2 * c) ^ z) << 4), pk[0], pk[1], pk[2], pk[3]);
          st_shared_v4(srow + (((2 * c + 1) ^ z) << 4), pk[4], pk[5], pk[6], pk[7]);
        }
        __syncwarp();
        const int u = lane % kUnits;  // 16-byte unit of the row this lane stores
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int r = i * (32 / kUnits) + lane / kUnits;  // row within the warp's 32
          const uint4 val = ld_shared_v4(
              stage + static_cast<uint32_t>(r * kHalf * 2 + ((u ^ (r & (kUnits - 1))) << 4)));
          const int row = quad * 32 + r;
          if (row < pc.rows) {
            const int tk = token_of(row);
            const long long at = static_cast<long long>(pc.row0 + tk) * args.H + head + (row - tk * args.G);
            *reinterpret_cast<uint4*>(args.o + at * D + kHalf * g + 8 * u) = val;
          }
        }
        if (t < pc.rows && g == 0) {
          const int tk = token_of(t);
          args.lse[static_cast<long long>(pc.row0 + tk) * args.H + head + (t - tk * args.G)] = lse2 * kLn2;
        }
      } else {
        // a piece: normalised, fp32. Slot 0 continues what an earlier CTA began, slot 1 is
        // continued by the next.
        const long long at = (2ll * blockIdx.x + (pc.from_start ? 1 : 0)) * kTile + t;
#pragma unroll
        for (int c = 0; c < kHalf / 16; ++c) {
          const uint32_t col = static_cast<uint32_t>(kHalf * g + 16 * c);
          uint32_t o0[16], o1[16];
          if (has0) tmem_ld16(tmem + lane_base + L::col_o(0) + col, o0);
          if (has1) tmem_ld16(tmem + lane_base + L::col_o(1) + col, o1);
          tmem_ld_wait();
          float y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            y[k] = has0 ? __uint_as_float(o0[k]) * w0 : 0.f;
            if (has1) y[k] = fmaf(__uint_as_float(o1[k]), w1, y[k]);
          }
          if (t < pc.rows) {
            float4* dst = reinterpret_cast<float4*>(args.o_part + at * D + col);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          }
        }
        if (t < pc.rows && g == 0) args.lse_part[at] = lse2;
      }
      if (tid == 0) {
        if (!pc.from_start) left->ended = pc.ends;
        if (pc.from_start && !pc.ends) {
          left->row0 = pc.row0;
          left->h = pc.h;
          left->rows = pc.rows;
        }
      }
      tc_fence_before();
      mbar_arrive(bars.o_free);
      __syncwarp();
      if (lane == 0) leave_piece(count);
      ++count;
      tile_cnt += nt;
      q_cnt += nt > 0;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of the pieces of a query tile that runs' ends have cut, a warp per row: with lse_s
// and the normalised O_s of piece s, O = sum_s 2^(lse_s - m) O_s / sum_s 2^(lse_s - m), m =
// max_s lse_s, in the order of the pieces. Blocks (c, ..) take the tile that CTA c's run
// began and did not end. A piece whose lse is a NaN takes no part in the maximum, and makes
// the sums NaN.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    fa_paged_chunk_merge_kernel(const PagedAttnArgs a, int ctas) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  __shared__ int n_more;
  pdl_wait();
  const PieceHeader* headers = static_cast<const PieceHeader*>(a.headers);
  PieceHeader hd;
  const int n = 1 + pieces_after(headers, c, ctas, &n_more, &hd);  // slot 1 of c, slot 0 of the others
  const int G = a.G;
  const int r = blockIdx.y * kMergeWarps + warp;
  if (hd.row0 < 0 || r >= hd.rows) return;
  auto row_of = [&](int i) { return (2ll * (c + i) + (i == 0 ? 1 : 0)) * kTile + r; };
  // the first pieces are under way while the maximum is found
  float m = -INFINITY, den = 0.f, acc[kPer] = {}, lse0[2] = {-INFINITY, -INFINITY}, part0[2][kPer] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i < n) {
      lse0[i] = a.lse_part[row_of(i)];
      load_part<kPer>(a.o_part + row_of(i) * D + lane * kPer, part0[i]);
    }
  }
  for (int i = lane; i < n; i += 32) m = fmaxf(m, a.lse_part[row_of(i)]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float mu = m == -INFINITY ? 0.f : m;
  auto add = [&](float lse, const float* part) {
    const float w = ex2_approx(lse - mu);
    den += w;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] += w * part[k];
  };
  add(lse0[0], part0[0]);
  add(lse0[1], part0[1]);
#pragma unroll 4
  for (int i = 2; i < n; ++i) {
    float part[kPer];
    load_part<kPer>(a.o_part + row_of(i) * D + lane * kPer, part);
    add(a.lse_part[row_of(i)], part);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int t = r / G;
  const long long row = static_cast<long long>(hd.row0 + t) * a.H + hd.h * G + (r - t * G);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + row * D + lane * kPer);
  dst[0] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if constexpr (kPer == 4) dst[1] = pack_bf16x2(acc[2] * inv, acc[3] * inv);
  if (lane == 0) a.lse[row] = den == 0.f ? -INFINITY : (m + __log2f(den)) * kLn2;
}

namespace {

template <int D, bool E4M3>
cudaError_t launch_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const PagedAttnArgs& a, int box_rows, int ctas, cudaStream_t stream) {
  using L = ChunkL<D, E4M3>;
  auto kern = fa_paged_chunk_kernel<D, E4M3>;
  // The in-kernel register reallocation assumes kRegsLaunch registers per thread at launch:
  // with fewer, the softmax warpgroups' increase could never be granted and would wait
  // forever, so such a kernel is refused.
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(kern), L::kSmemBytes, L::kRegsLaunch, ready);
  if (e != cudaSuccess) return e;
  kern<<<ctas, L::kThreads, L::kSmemBytes, stream>>>(tq, tk, tv, a, box_rows);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_merge(fa_paged_chunk_merge_kernel<D>, dim3(ctas, kTile / kMergeWarps),
                      kMergeWarps * 32, stream, a, ctas);
}

}  // namespace

cudaError_t launch_paged_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, bool e4m3, int box_rows, int ctas,
                               cudaStream_t stream) {
  if (a.c.d == 64)
    return e4m3 ? launch_impl<64, true>(tq, tk, tv, a, box_rows, ctas, stream)
                : launch_impl<64, false>(tq, tk, tv, a, box_rows, ctas, stream);
  return e4m3 ? launch_impl<128, true>(tq, tk, tv, a, box_rows, ctas, stream)
              : launch_impl<128, false>(tq, tk, tv, a, box_rows, ctas, stream);
}

}  // namespace fa
