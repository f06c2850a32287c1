// Shared device-side pieces of the attention kernels: launch parameters,
// tile validity (causal / key padding / block-sparse), the Philox dropout
// generator and the device status word.
#pragma once
#include <climits>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace fa {

constexpr int kTile = 128;               // query / key tile edge (rows), and block-mask granularity
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Device status codes (mirror fa_status in include/fa.h).
constexpr unsigned kStatusCuda = 3u;     // a launch found its configuration unusable
constexpr unsigned kStatusTimeout = 5u;

// A run of consecutive mbarriers (8 bytes each) addressed by index. An array of
// barrier addresses indexed by a ring stage would be placed in local memory, so
// every handshake would first load its barrier's address from there.
struct BarRun {
  uint32_t base;
  __device__ __forceinline__ uint32_t operator[](int i) const {
    return base + 8u * static_cast<uint32_t>(i);
  }
};

// Instances of the bf16 forward and backward kernels. kPlain and kWindow have as many queries as
// keys. kCross has Nq queries at positions q_off .. of an axis of Nk keys, with every mask but the
// block mask; kRel adds a bias by relative position to it.
enum Mode : int { kPlain = 0, kWindow = 1, kCross = 2, kRel = 3 };

struct MaskParams {
  int B, H, N;                  // N: query rows (and keys, but for kCross and kRel)
  int Hkv;                      // K/V heads (H for per-head attention; H / Hkv query heads share one)
  int nb;                       // ceil(N / 128): tiles per side, block-mask row length
  int causal;
  int wl, wr;                   // sliding window: keys i - wl .. i + wr visible (-1: unbounded)
  const uint8_t* block_mask;    // [nb, nb] or null
  const int32_t* seqlens_k;     // [B] or null
  int Nk;                       // keys
  int q_off;                    // kCross, kRel: query i sits at position i + q_off of the key axis
};

// The bias of the scores by relative position (kRel): the distance of key j from the query at
// position p is j - p, and what lies beyond -left and right counts as these. Each head has a line
// of its biases in log2 units, by distance from -left - kRelPad to right + kRelPad, so that the
// distances of a tile that is not wholly beyond an end (at most 253 past it) need no clamp. Behind
// the line lie its windows, for each distance the biases of it and the next three: a thread's
// biases begin at any distance, and four of them are one aligned load; a warp's are 35 windows in a
// row. (Forward of B=4 H=8 N=2000 d=128, range 1000: 94 us, with a load per bias 102, with four
// copies of the line that begin one distance apart 116.)
constexpr int kRelPad = 256;
struct RelParams {
  const float* lines;           // [H, pitch + 4 pitch], 16-byte aligned
  int left, right;
  __host__ __device__ int pitch() const { return (left + right + 1 + 2 * kRelPad + 3) & ~3; }
  __host__ __device__ int stride() const { return 5 * pitch(); }
};

// Where a block of n queries x n keys lies whose first key is d0 behind its first query: its
// distances are d0 - (n - 1) .. d0 + (n - 1). Beyond an end of the range the bias is one number.
__device__ __forceinline__ bool rel_far_left(const RelParams& r, int d0, int n = kTile) {
  return d0 + (n - 1) <= -r.left;
}
__device__ __forceinline__ bool rel_far_right(const RelParams& r, int d0, int n = kTile) {
  return d0 - (n - 1) >= r.right;
}

__device__ __forceinline__ bool rel_far(const RelParams& r, int d0) {
  return rel_far_left(r, d0) || rel_far_right(r, d0);
}

// The line of head h, indexed by distance.
__device__ __forceinline__ const float* rel_line(const RelParams& r, int h) {
  return r.lines + static_cast<size_t>(h) * r.stride() + r.left + kRelPad;
}

// The bias of a head: its line, and the biases beyond the ends.
struct RelHead {
  const float* line;
  float left, right;
};
__device__ __forceinline__ RelHead rel_head(const RelParams& r, int h) {
  RelHead x;
  x.line = rel_line(r, h);
  x.left = __ldg(x.line - r.left);
  x.right = __ldg(x.line + r.right);
  return x;
}

// Bias of a block beyond an end of the range (0 for others, whose elements have their own).
__device__ __forceinline__ float rel_far_bias(const RelParams& r, const RelHead& x, int d0,
                                              int n = kTile) {
  return rel_far_left(r, d0, n) ? x.left : (rel_far_right(r, d0, n) ? x.right : 0.f);
}

// Windows of four biases of a head, by the distance of the first.
__device__ __forceinline__ const float4* rel_windows(const RelParams& r, const float* line) {
  return reinterpret_cast<const float4*>(line - r.left - kRelPad + r.pitch()) + r.left + kRelPad;
}

// Adds to N scores of this thread their own biases and brings them to log2 units: the first one's
// is at distance dist, the others STEP apart. AT_ONCE of them are loaded together (more cost the
// backward kernels registers; with 8 at a time the forward above takes 110 us).
template <int N, int STEP, int AT_ONCE>
__device__ __forceinline__ void rel_add(const RelParams& r, const float* line, int dist,
                                        float c_log2, float* s) {
  static_assert(STEP == 1 || STEP == -1, "keys or queries in order");
  const uint64_t c2 = f2_pack(c_log2, c_log2);
  const float4* lp = rel_windows(r, line) + (STEP == 1 ? dist : dist - 3);
#pragma unroll
  for (int i = 0; i < N; i += AT_ONCE) {
    float4 b[AT_ONCE / 4];
#pragma unroll
    for (int k = 0; k < AT_ONCE / 4; ++k) b[k] = __ldg(lp + STEP * (i + 4 * k));
#pragma unroll
    for (int k = 0; k < AT_ONCE / 4; ++k) {
      float* x = s + i + 4 * k;
      const uint64_t lo = STEP == 1 ? f2_pack(b[k].x, b[k].y) : f2_pack(b[k].w, b[k].z);
      const uint64_t hi = STEP == 1 ? f2_pack(b[k].z, b[k].w) : f2_pack(b[k].y, b[k].x);
      f2_unpack(f2_fma(f2_pack(x[0], x[1]), c2, lo), x[0], x[1]);
      f2_unpack(f2_fma(f2_pack(x[2], x[3]), c2, hi), x[2], x[3]);
    }
  }
}

struct DropParams {
  int p8;                       // drop iff Philox byte < p8
  float keep_scale;             // 1 / (1 - p8 / 256)
  uint32_t seed_lo, seed_hi, off_lo, off_hi;
  // Philox round keys, (seed_lo + r W0, seed_hi + r W1) mod 2^32 for rounds
  // r = 0..9, filled on the host so that a kernel reads them as constant
  // operands instead of bumping the key every round. Pairs on 16-byte boundaries: dQ of H=16
  // N=16384 d=64 takes 2454 us; as two arrays 2533 to 2555, by where they happen to begin.
  alignas(16) uint2 rk[10];
};

struct SyncParams {
  unsigned int* status;         // device status word (first error wins)
  unsigned long long timeout_ns;
  int inject_stall;             // test hook: wait on a barrier that never completes
};

__device__ __forceinline__ void record_error(unsigned int* status, unsigned code) {
  atomicCAS(status, 0u, code);
}

// K/V head of query head bh = b*H + h: grouped-query attention gives the H / Hkv
// query heads h of a group the K/V head h / (H / Hkv) of the same batch row.
__device__ __forceinline__ int kv_head(const MaskParams& m, int bh) {
  const int b = bh / m.H, h = bh - b * m.H;
  return b * m.Hkv + h / (m.H / m.Hkv);
}

// First query head bh = b*H + h of the group that shares K/V head bhk = b*Hkv + j;
// the group is the G = H / Hkv consecutive heads from there. With one query head
// per K/V head (GQA false) that is bhk itself.
template <bool GQA>
__device__ __forceinline__ int group_first_head(const MaskParams& m, int bhk) {
  if constexpr (!GQA) return bhk;
  return (bhk / m.Hkv) * m.H + (bhk % m.Hkv) * (m.H / m.Hkv);
}

// Number of valid keys of batch b (key padding clamps to [0, Nk]).
__device__ __forceinline__ int kv_len_of(const MaskParams& m, int b) {
  if (m.seqlens_k == nullptr) return m.Nk;
  int L = m.seqlens_k[b];
  return L < 0 ? 0 : (L > m.Nk ? m.Nk : L);
}

// kCross, kRel: position of the first row of query tile qt on the key axis.
__device__ __forceinline__ int tile_pos(const MaskParams& m, int qt) {
  return qt * kTile + m.q_off;
}

// Key tiles [0, bound) hold every tile that is valid for query tiles .. qt_end - 1: n_kv, or with
// a causal mask those up to the last row's position.
template <int MODE>
__device__ __forceinline__ int key_tiles_upto(const MaskParams& m, int qt_end, int n_kv) {
  int bound = n_kv;
  if constexpr (MODE >= kCross) {
    if (m.causal) {
      const int end = tile_pos(m, qt_end);  // positions below it are reached
      const int c = end > 0 ? (end - 1) / kTile + 1 : 0;
      if (c < bound) bound = c;
    }
  } else {
    if (m.causal && qt_end < bound) bound = qt_end;
  }
  return bound;
}

// kCross, kRel with key lengths: batch rows in falling order of their number of key tiles, so that
// the alternation of sched_unit gives every CTA long units and short ones, the short ones last.
// (Rows of a batch that is not ordered come as they are: more than kMaxOrdered make units enough.
// With the list of key tiles of the dK/dV kernel, 448 queries over 300 to 1500 keys, B=16 H=16 d=64:
// forward and backward 243 us, without either 293.)
constexpr int kMaxOrdered = 256;
__device__ __forceinline__ bool is_ordered(const MaskParams& m) {
  return m.seqlens_k != nullptr && m.B > 1 && m.B <= kMaxOrdered;
}
__device__ __forceinline__ void order_by_length(const MaskParams& m, uint8_t* order, int tid,
                                                int threads) {
  if (!is_ordered(m)) return;
  for (int b = tid; b < m.B; b += threads) {
    const int n = (kv_len_of(m, b) + kTile - 1) / kTile;
    int rank = 0;
    for (int i = 0; i < m.B; ++i) {
      const int x = (kv_len_of(m, i) + kTile - 1) / kTile;
      rank += (x > n || (x == n && i < b)) ? 1 : 0;
    }
    order[rank] = static_cast<uint8_t>(b);
  }
}
// Head b*H + h at position x of the heads in that order.
__device__ __forceinline__ int ordered_head(const MaskParams& m, const uint8_t* order, int x) {
  if (!is_ordered(m)) return x;
  const int s = x / m.H;
  return order[s] * m.H + (x - s * m.H);
}

// Static schedule of the persistent kernels: in round k the CTAs take the
// positions [k G, k G + G) of the work list, G = gridDim.x, in forward order
// on even rounds and in reverse order on odd rounds. Every role of a CTA walks
// the same sequence. With a causal mask the work list is ordered longest unit
// first within each head, so a CTA that drew a long unit in one round draws a
// short one in the next and the per-CTA totals stay within a few percent of
// each other; head-major order keeps the CTAs of a round on a few heads, whose
// K/V tiles they then share in L2. Returns a position >= the list length once
// the CTA has no more work (positions grow with k).
// With rotate set, round k instead shifts the positions by k: the dK/dV work
// list under key padding has its empty units (key tiles past a batch row's
// length) at the same places in every head, so the alternation would hand some
// CTAs a key tile and its mirror, both often empty, in every round, and others
// none; rotating lets every CTA meet every key tile.
__device__ __forceinline__ int sched_unit(int k, bool rotate = false) {
  const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  if (rotate) return k * G + (c + k) % G;
  return k * G + ((k & 1) ? (G - 1 - c) : c);
}

// Whether the (query tile qt, key tile kt) pair has any allowed element.
// n_kv = ceil(kv_len / 128), n_q = ceil(N / 128). With a sliding window (a
// separate kernel instance, so that kernels without one keep their code)
// the pair is skipped when the band i - wl <= j <= i + wr misses the tile.
template <int MODE = kPlain>
__device__ __forceinline__ bool tile_valid(const MaskParams& m, int qt, int kt, int n_q,
                                           int n_kv) {
  if (qt >= n_q || kt >= n_kv) return false;
  if constexpr (MODE >= kCross) {
    const int p0 = tile_pos(m, qt), k0 = kt * kTile;
    if (m.causal && k0 > p0 + (kTile - 1)) return false;
    if (m.wl >= 0 && k0 + (kTile - 1) + m.wl < p0) return false;
    if (m.wr >= 0 && k0 > p0 + (kTile - 1) + m.wr) return false;
    return true;
  }
  if (m.causal && kt > qt) return false;
  if constexpr (MODE == kWindow) {
    if (m.wl >= 0 && kt * kTile + (kTile - 1) + m.wl < qt * kTile) return false;
    if (m.wr >= 0 && kt * kTile > qt * kTile + (kTile - 1) + m.wr) return false;
  }
  if (m.block_mask != nullptr && m.block_mask[qt * m.nb + kt] == 0) return false;
  return true;
}

// Whether the pair needs a per-element mask (causal diagonal, key tile
// crossing kv_len, or a sliding-window edge inside the tile). Query rows
// beyond N are never written, so the query tail needs none.
template <int MODE = kPlain>
__device__ __forceinline__ bool tile_needs_element_mask(const MaskParams& m, int qt, int kt,
                                                        int kv_len) {
  if constexpr (MODE >= kCross) {
    const int p0 = tile_pos(m, qt), k0 = kt * kTile;
    return (m.causal && k0 + (kTile - 1) > p0) || (m.wl >= 0 && k0 < p0 + (kTile - 1) - m.wl) ||
           (m.wr >= 0 && k0 + (kTile - 1) > p0 + m.wr) || k0 + kTile > kv_len;
  }
  if constexpr (MODE == kWindow) {
    if (m.wl >= 0 && kt * kTile < qt * kTile + (kTile - 1) - m.wl) return true;
    if (m.wr >= 0 && kt * kTile + (kTile - 1) > qt * kTile + m.wr) return true;
  }
  return (m.causal && kt == qt) || ((kt + 1) * kTile > kv_len);
}

// A run of tiles [lo, hi).
struct TileRun {
  int lo, hi;
  __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
};
__device__ __forceinline__ int floor_tiles(int x) { return x >> 7; }         // x / 128 rounded down
__device__ __forceinline__ int ceil_tiles(int x) { return (x + 127) >> 7; }  // and up
static_assert(kTile == 128, "shifts by 7");

// kCross, kRel: the key tiles of a query tile whose first row is at position p0 (the query tiles of
// key tile kt) that need no mask per element.
__device__ __forceinline__ TileRun free_key_tiles(const MaskParams& m, int p0, int kv_len) {
  TileRun r{0, floor_tiles(kv_len)};
  if (m.causal) r.hi = min(r.hi, floor_tiles(p0 + 1));
  if (m.wr >= 0) r.hi = min(r.hi, floor_tiles(p0 + m.wr + 1));
  if (m.wl >= 0) r.lo = ceil_tiles(p0 + (kTile - 1) - m.wl);
  return r;
}
__device__ __forceinline__ TileRun free_query_tiles(const MaskParams& m, int kt, int kv_len) {
  const int k0 = kt * kTile - m.q_off;
  TileRun r{0, INT_MAX};
  if (m.causal) r.lo = ceil_tiles(k0 + kTile - 1);
  if (m.wr >= 0) r.lo = max(r.lo, ceil_tiles(k0 + kTile - 1 - m.wr));
  if (m.wl >= 0) r.hi = floor_tiles(k0 - (kTile - 1) + m.wl) + 1;
  if ((kt + 1) * kTile > kv_len) r.hi = 0;
  return r;
}

// kCross, kRel: the query tiles that see some key of key tile kt (tile_valid).
__device__ __forceinline__ TileRun seeing_query_tiles(const MaskParams& m, int kt, int n_q) {
  TileRun r{0, n_q};
  const int k0 = kt * kTile - m.q_off;
  if (m.causal) r.lo = max(r.lo, ceil_tiles(k0 - (kTile - 1)));
  if (m.wr >= 0) r.lo = max(r.lo, ceil_tiles(k0 - m.wr - (kTile - 1)));
  if (m.wl >= 0) r.hi = min(r.hi, floor_tiles(k0 + (kTile - 1) + m.wl) + 1);
  return r;
}

// kCross, kRel: the key tiles that a query tile at position p0 sees some key of (tile_valid).
__device__ __forceinline__ TileRun seen_key_tiles(const MaskParams& m, int p0, int n_kv) {
  TileRun r{0, n_kv};
  if (m.causal) r.hi = min(r.hi, floor_tiles(p0 + kTile - 1) + 1);
  if (m.wr >= 0) r.hi = min(r.hi, floor_tiles(p0 + kTile - 1 + m.wr) + 1);
  if (m.wl >= 0) r.lo = max(0, ceil_tiles(p0 - m.wl - (kTile - 1)));
  return r;
}

// kRel: the tiles along one axis whose block of n queries x n keys lies within reach of the
// diagonal, at distance d0 + 128 i for key tile i: before them it is far to the left, behind them
// far to the right.
__device__ __forceinline__ TileRun near_tiles(const RelParams& r, int d0, int n = kTile) {
  // not d0 + 128 i + n - 1 <= -left, and not d0 + 128 i - (n - 1) >= right
  return TileRun{floor_tiles(-r.left - (n - 1) - d0) + 1, ceil_tiles(r.right + (n - 1) - d0)};
}

// The same for the query tiles of key tile kt: distance kt * 128 - q_off - 128 i for query tile i.
__device__ __forceinline__ TileRun near_query_tiles(const RelParams& r, const MaskParams& m, int kt) {
  const int d0 = kt * kTile - m.q_off;
  return TileRun{floor_tiles(d0 - (kTile - 1) - r.right) + 1, ceil_tiles(d0 + (kTile - 1) + r.left)};
}

// kCross, kRel: keys [lo, lim) of key tile kt, counted from its first, are visible to the query at
// position pos.
__device__ __forceinline__ void visible_keys(const MaskParams& m, int pos, int kt, int kv_len,
                                             int& lo, int& lim) {
  const int k0 = kt * kTile;
  lim = kv_len - k0;
  lo = 0;
  if (m.causal) lim = min(lim, pos + 1 - k0);
  if (m.wr >= 0) lim = min(lim, pos + m.wr + 1 - k0);
  if (m.wl >= 0) lo = pos - m.wl - k0;
}

// kCross, kRel: of the queries at positions pos0, pos0 + 1, .. those from lo to hi - 1 see key `key`.
__device__ __forceinline__ void seeing_queries(const MaskParams& m, int key, int pos0, int kv_len,
                                               int& lo, int& hi) {
  lo = 0;
  hi = kTile;
  if (m.causal) lo = key - pos0;
  if (m.wr >= 0) lo = max(lo, key - m.wr - pos0);
  if (m.wl >= 0) hi = min(hi, key + m.wl - pos0 + 1);
  if (key >= kv_len) hi = 0;
}

// kCross, kRel: the key tile that a length below Nk cuts (-1: none) has rows behind it, which may
// hold anything; a weight of zero does not keep a NaN or an infinity there out of a product.
// (Rows from Nk on arrive as zeros.)
__device__ __forceinline__ int cut_tile(const MaskParams& m, int kv_len) {
  return kv_len < m.Nk && kv_len % kTile != 0 ? kv_len / kTile : -1;
}

// Zeroes rows [first, 128) of a 128 x (64 CHUNKS) bf16 tile in shared memory, with `n` threads of
// which this is thread i, and makes that visible to the tensor core's reads.
template <int CHUNKS>
__device__ __forceinline__ void zero_tile_rows(uint32_t tile, int first, int i, int n) {
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)  // (a row's 128 bytes are permuted within themselves)
    for (int u = first * 8 + i; u < kTile * 8; u += n)
      st_shared_v4(tile + static_cast<uint32_t>(c * 16384 + u * 16), 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
}

// Whether key j is inside query i's sliding window.
__device__ __forceinline__ bool in_window(const MaskParams& m, int i, int j) {
  return (m.wl < 0 || j >= i - m.wl) && (m.wr < 0 || j <= i + m.wr);
}

// Bits j in [32*c, 32*c + 32) that are valid for query tile qt, computed by a
// whole warp (one candidate per lane).
template <int MODE = kPlain>
__device__ __forceinline__ uint32_t warp_valid_bits(const MaskParams& m, int qt, int chunk,
                                                    int n_q, int n_kv) {
  const int lane = threadIdx.x & 31;
  const bool v = tile_valid<MODE>(m, qt, chunk * 32 + lane, n_q, n_kv);
  return __ballot_sync(0xffffffffu, v);
}

// Same, transposed: query tiles qt in [32*c, 32*c + 32) valid for key tile kt.
template <int MODE = kPlain>
__device__ __forceinline__ uint32_t warp_valid_bits_t(const MaskParams& m, int kt, int chunk,
                                                      int n_q, int n_kv) {
  const int lane = threadIdx.x & 31;
  const bool v = tile_valid<MODE>(m, chunk * 32 + lane, kt, n_q, n_kv);
  return __ballot_sync(0xffffffffu, v);
}

// ------------------------------------------------------------------ Philox
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy
// as 1, 2, 3", SC'11): ten rounds of two 32x32 -> 64-bit multiplies by the
// round multipliers, the high halves xored with the other counter words and
// the key, with the key advanced by the Weyl increments between rounds.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    if (r > 0) {
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    const uint32_t lo0 = 0xD2511F53u * c.x;
    const uint32_t hi0 = __umulhi(0xD2511F53u, c.x);
    const uint32_t lo1 = 0xCD9E8D57u * c.z;
    const uint32_t hi1 = __umulhi(0xCD9E8D57u, c.z);
    c = make_uint4(hi1 ^ c.y ^ k0, lo1, hi0 ^ c.w ^ k1, lo0);
  }
  return c;
}

// The same generator with the round keys taken from DropParams.
__device__ __forceinline__ uint4 philox4x32_10_rk(uint4 c, const DropParams& d) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    // one widening multiply gives both halves of each 64-bit product
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c.x;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
    const uint32_t lo0 = static_cast<uint32_t>(p0), hi0 = static_cast<uint32_t>(p0 >> 32);
    const uint32_t lo1 = static_cast<uint32_t>(p1), hi1 = static_cast<uint32_t>(p1 >> 32);
    c = make_uint4(hi1 ^ c.y ^ d.rk[r].x, lo1, hi0 ^ c.w ^ d.rk[r].y, lo0);
  }
  return c;
}

// Byte permute: result byte i = byte sel.nibble[i] of the 8-byte value {b, a}
// (a = bytes 0-3); a nibble with bit 3 set replicates that byte's sign bit.
// Used to turn dropout keep bytes (0x00 / 0xFF) into lane masks.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Keep masks for the 16 keys [16*g, 16*g + 16) of query row `row_global`
// ((b*H + h)*N + i): each byte is 0xFF where the element is kept, 0 where dropped.
__device__ __forceinline__ uint4 dropout_keep16(const DropParams& d, uint32_t row_global,
                                                uint32_t key_group) {
  const uint4 r = philox4x32_10_rk(make_uint4(key_group, row_global, d.off_lo, d.off_hi), d);
  const uint32_t thr = static_cast<uint32_t>(d.p8) * 0x01010101u;
  // Per-byte unsigned compare x >= p8 in SWAR form: the subtraction of the low
  // seven bits cannot borrow across bytes (bit 7 of each minuend byte is set),
  // so bit 7 of each byte of dif is [low7(x) >= low7(p8)]; x >= p8 when x's
  // top bit is set and p8's is not, or when they agree and dif's is set. The
  // byte permute then spreads each byte's top bit to 0xFF or 0x00.
  auto ge = [thr](uint32_t x) {
    const uint32_t dif = (x | 0x80808080u) - (thr & 0x7F7F7F7Fu);
    const uint32_t top = (x & ~thr) | (~(x ^ thr) & dif);
    return prmt(top, 0u, 0xBA98u);
  };
  return make_uint4(ge(r.x), ge(r.y), ge(r.z), ge(r.w));
}

// bf16x2 helpers for the epilogues.
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) { return pack_bf16x2(lo, hi); }

}  // namespace fa
