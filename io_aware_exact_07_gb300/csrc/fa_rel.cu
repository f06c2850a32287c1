// Learned relative position bias: the lines of biases that the attention kernels read, and the
// gradient of the table they come from.
//
// The score of key j for the query at position p gets table[map[clamp(j - p, -left, right) + left],
// h]. A head's biases by distance form one line, which is a few KB for the usual rules, so the
// attention kernels read it from L1 or add one number to a whole tile that lies beyond an end of
// the range. The gradient of a table entry is the sum of dS over the pairs whose distance maps to
// it:
//   dS_ij = P_ij (Z_ij/(1-p) dO_i.v_j - D_i),  D_i = sum_j P_ij Z_ij/(1-p) dO_i.v_j.
// The backward kernels take D_i from the rounded O. That is off by up to 2^-9 |dO_i||O_i|, and a
// sum over many pairs of one row collects it: R_i = sum_j dS_ij would be zero with the exact D_i
// (the weights of a row sum to one), so D_i + R_i is the D of the unrounded O, and the sum of dS
// over a set of keys of the row is corrected by -R_i times their weights' sum. The dQ kernel
// leaves R_i and the sums of dS and P over the tiles beyond either end of the range:
//   rel_near    recomputes dS on the tiles near the diagonal, with D + R. For a fixed kt - qt every
//               tile has the same distance at the same place, so a CTA adds tiles of a head and
//               kt - qt, over batch rows and query tiles, element by element in registers and
//               forms the sums along the diagonals once, when it moves on;
//   rel_sums    adds the diagonals' sums up by distance, and the rows' sums of the two far fields;
//   rel_table   adds the distances and the far fields up by bucket.
// Sums are fp32, over few values each; the long ones at the end keep what each addition rounds off
// (Knuth's two-sum): this GPU adds fp64 at a 64th of the rate.
// No atomics: the order of every sum is fixed.
//
// The kernel of the near tiles also serves the backward pass of all calls with positions: for query
// tiles whose rows see one key tile it forms D_i itself, before the other kernels use it. There the
// rounding of O is most of what dQ and dK are off (5 keys: 0.37 % of dQ; with the D of the scores
// 0.24 % are left, as with many keys).
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
#include "fa_kernels.h"
#include "fa_launch.cuh"

namespace fa {

namespace {

constexpr unsigned kStatusInvalid = 1u;
constexpr float kRelMaxBias = 32768.f;  // entries of a table

__device__ __forceinline__ int clamp_distance(int x, int left, int right) {
  return x < -left ? -left : (x > right ? right : x);
}

// A sum with its rounding errors.
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& x) {
    add(x.hi);
    lo = __fadd_rn(lo, x.lo);
  }
  // over the warp; the same on every lane
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Sum x;
      x.hi = __shfl_xor_sync(0xffffffffu, hi, o);
      x.lo = __shfl_xor_sync(0xffffffffu, lo, o);
      add(x);
    }
  }
};

// ------------------------------------------------------------------ lines
__global__ void __launch_bounds__(256) rel_lines_kernel(const RelLinesArgs a) {
  const RelParams r{nullptr, a.left, a.right};
  const int e = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y;
  if (e >= r.stride()) return;
  const int w = e - r.pitch();  // of the windows
  const int dist = (w < 0 ? e : (w >> 2) + (w & 3)) - a.left - kRelPad;
  const int n = __ldg(a.map + clamp_distance(dist, a.left, a.right) + a.left);
  float x = 0.f;
  if (n < 0 || n >= a.num_buckets) {
    record_error(a.status, kStatusInvalid);
  } else {
    const size_t at = static_cast<size_t>(n) * a.H + h;
    x = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.table)[at])
               : static_cast<const float*>(a.table)[at];
    // fp32 scores and lse tell keys of such a bias apart to 2^-9 (a weight to less than the half step
    // of bf16 that it is rounded by), and worse beyond: lower entries hide, higher ones are refused
    if (x <= -kRelMaxBias) x = -INFINITY;
    if (x > kRelMaxBias) {
      record_error(a.status, kStatusInvalid);
      x = kRelMaxBias;
    }
  }
  a.lines[static_cast<size_t>(h) * r.stride() + e] = x * kLog2e;
}

// ------------------------------------------------------------------ rows
// One block takes kRelRows query rows of a head (b, h).
__device__ __forceinline__ void rows_sums(const RelGradArgs& a, int chunks, int block) {
  const int bh = block / chunks, chunk = block % chunks, N = a.b.mask.N;
  const size_t rows = static_cast<size_t>(a.b.mask.B) * a.b.mask.H * N;
  float left = 0.f, right = 0.f;
  static_assert(kRelRows == 256, "a thread per row");
  const int row = chunk * kRelRows + static_cast<int>(threadIdx.x);
  if (row < N) {
    const size_t idx = static_cast<size_t>(bh) * N + row;
    float s[kRelRowSums];
#pragma unroll
    for (int k = 0; k < kRelRowSums; ++k) {
      const float* p = a.b.row_sums + 4 * rows * k + idx;
      s[k] = (p[0] + p[rows]) + (p[2 * rows] + p[3 * rows]);
    }
    // (a row that sees no key has sums of zero)
    left = fmaf(-s[0], 1.f - s[3], s[1]);
    right = fmaf(-s[0], s[4], s[2]);
  }
  __shared__ float part[2][8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    left += __shfl_xor_sync(0xffffffffu, left, o);
    right += __shfl_xor_sync(0xffffffffu, right, o);
  }
  if ((threadIdx.x & 31) == 0) {
    part[0][threadIdx.x >> 5] = left;
    part[1][threadIdx.x >> 5] = right;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const float* x = part[threadIdx.x];
    a.far_sums[static_cast<size_t>(block) * 2 + threadIdx.x] =
        ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  }
}

// ------------------------------------------------------------------ near tiles
// The list of near tile pairs: by head, then kt - qt (a group of pairs has one of each), then
// batch row, then query tile. CTA c takes per_cta of them from c * per_cta on.
struct NearList {
  int n_q, n_k, B, first, n_diag;
  __device__ int begin(int g) const { return max(0, -(first + g)); }  // query tiles of kt - qt
  __device__ int count(int g) const { return max(0, min(n_q, n_k - (first + g)) - begin(g)); }
  __device__ long long head_total() const {
    long long n = 0;
    for (int g = 0; g < n_diag; ++g) n += count(g);
    return n * B;
  }
};

__device__ __forceinline__ NearList near_list(const RelGradArgs& a) {
  NearList l;
  l.n_q = (a.b.mask.N + kTile - 1) / kTile;
  l.n_k = (a.b.mask.Nk + kTile - 1) / kTile;
  l.B = a.b.mask.B;
  l.first = a.first;
  l.n_diag = a.n_diag;
  return l;
}

__device__ __forceinline__ long long near_per_cta(long long total, int ctas) {
  return (total + ctas - 1) / ctas;
}

// A walk over the pairs of one CTA.
struct NearWalk {
  NearList l;
  long long left;  // pairs from here on, this one included
  int h, g, b, i;  // head, group of the head, batch row, query tile counted from the group's first
  int n;           // query tiles of the group

  __device__ NearWalk(const NearList& list, int H, int ctas, int cta) : l(list) {
    left = h = g = b = i = n = 0;
    if (ctas == 0) return;
    const long long per_head = l.head_total(), total = per_head * H;
    const long long per = near_per_cta(total, ctas), at = per * cta;
    left = max(0ll, min(per, total - at));
    if (left == 0) return;
    h = static_cast<int>(at / per_head);
    long long rest = at % per_head;
    while (rest >= static_cast<long long>(l.count(g)) * l.B) {
      rest -= static_cast<long long>(l.count(g)) * l.B;
      ++g;
    }
    n = l.count(g);
    b = static_cast<int>(rest / n);
    i = static_cast<int>(rest % n);
  }
  __device__ int qt() const { return l.begin(g) + i; }
  __device__ int kt() const { return qt() + l.first + g; }
  __device__ int group() const { return h * l.n_diag + g; }
  __device__ void next() {
    --left;
    if (++i < n) return;
    i = 0;
    if (++b < l.B) return;
    b = 0;
    do {
      if (++g == l.n_diag) {
        g = 0;
        ++h;
      }
      n = l.count(g);
    } while (n == 0 && left > 0);
  }
};

constexpr int kNearComputeWarps = 16;
constexpr int kNearCompute = kNearComputeWarps * 32;
constexpr int kNearProducerWarp = 16;
constexpr int kNearMmaWarp = 17;
constexpr int kNearThreads = 18 * 32;
constexpr int kDiagPitch = 33;
// The producer walks the list and hands each pair on in shared memory: head b*H + h (-1: no more),
// query tile, key tile, group; key length and the CTA's first group. Pair n's slot is taken again
// for pair n + 8, whose ring stage pair n + 5 or a later one has left: its products waited until
// the compute warps had read the S of pair n + 3, and they read the slot of a pair before the S of
// the one in front of it.
constexpr int kPairSlots = 8;

template <int D>
struct NearL {
  static constexpr int T = kTile * D * 2;
  static constexpr int kChunks = D / 64;
  static constexpr int kStages = D == 64 ? 6 : 3;  // ring of tile pairs: (Q, K), (dO, V), ...
  static constexpr int kDiagOff = kStages * 2 * T;
  static constexpr int kLineOff = kDiagOff + 2 * kTile * kDiagPitch * 4;
  static constexpr int kBarOff = kLineOff + 256 * 4;
  static constexpr int kNumBars = 2 * kStages + 4 + kPairSlots + 1 + 5 + 4;
  static constexpr int kPairOff = kBarOff + (kNumBars + 1) / 2 * 16;
  static constexpr int kMiscOff = kPairOff + kPairSlots * 32;
  // no slack for rounding the base up: the kernel checks its alignment
  static constexpr int kSmemBytes = kMiscOff + 16;
  static_assert(kSmemBytes <= 232448, "shared memory exceeds the per-block limit");
};

// What bounds it: a pair of tiles takes 1.6 us at either head size (B=16 H=16 N=1024 d=64, 5632 pairs,
// 62 us; 2000 keys, 2001 distances, d=128, 6400 pairs: 68), where its products need 0.06 (d = 64), its
// exponentials 0.5 and its bytes from L2 0.5. The tensor pipe is active 11 % of cycles, warps issue in 46 %:
// it is each warp's chain from the wait for S over two loads from tensor memory to the sums. Loading
// the biases four at a time gained 1 us, forming the diagonals' sums in four parts 2.
// ROWS: instead of the near pairs' sums, D of the rows that see one key tile (launch_row_d).
// Only warpgroup 0 waits for the others' sums, and the biases come from the windows (each tile's
// distances differ): 2.0 us a tile, with all waiting for all 2.35 (B=7 H=16, 6763 queries, 95 keys).
template <int D, bool DROPOUT, bool ROWS>
__global__ void __launch_bounds__(kNearThreads, 1)
    rel_near_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_do, const RelGradArgs args) {
  using L = NearL<D>;
  constexpr int T = L::T;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {  // uniform over the block: nothing has started yet
    if (threadIdx.x == 0) record_error(args.b.sync.status, kStatusCuda);
    return;
  }
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const MaskParams& mk = args.b.mask;
  const int N = mk.N;

  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff + 8);
  const BarRun full{smem_u32(bar_mem)};                          // ring stages
  const BarRun empty{full.base + 8u * L::kStages};
  const BarRun s_full{empty.base + 8u * L::kStages};             // S and dP buffers
  const BarRun s_free{s_full.base + 16u};
  const BarRun pair_full{s_free.base + 16u};
  const uint32_t drain = pair_full.base + 8u * kPairSlots;
  const BarRun meet{drain + 8u};  // the compute warps; then each warpgroup
  const BarRun summed{meet.base + 40u};  // ROWS: the warpgroups' sums of pair n are in part n % 4
  int4* pairs = reinterpret_cast<int4*>(smem + L::kPairOff);
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full[s], 1);
      mbar_init(empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full[x], 1);
      mbar_init(s_free[x], kNearCompute);
    }
    for (int s = 0; s < kPairSlots; ++s) mbar_init(pair_full[s], 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 5; ++i) mbar_init(meet[i], i == 0 ? kNearCompute : 128);
    for (int i = 0; i < 4; ++i) mbar_init(summed[i], kNearCompute);
    fence_mbar_init();
  }
  if (warp == kNearMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = args.b.sync.timeout_ns;
  auto fail = [&]() {
    *abort_flag = 1;
    record_error(args.b.sync.status, kStatusTimeout);
  };
  const uint32_t sRing = smem_u32(smem);

  if (warp == kNearProducerWarp) {
    if (lane == 0) {
      const NearList list = near_list(args);
      NearWalk w(list, mk.H, ROWS ? 0 : gridDim.x, blockIdx.x);
      const int first_group = w.left > 0 ? w.group() : -1;
      uint32_t it = 0;
      bool ok = true;
      int group = -1;
      // the ring's next stage, and the slot of the pair that it begins
      auto hand_on = [&](int bh, int qt, int kt, int kv_len) -> bool {
        const int s = it % L::kStages;
        if (!mbar_wait(empty[s], ((it / L::kStages) & 1u) ^ 1u, tmo, abort_flag)) return false;
        const uint32_t slot = (it >> 1) % kPairSlots;
        pairs[2 * slot] = make_int4(bh, qt, kt, group);
        pairs[2 * slot + 1] = make_int4(kv_len, first_group, 0, 0);
        mbar_arrive(pair_full[slot]);
        return true;
      };
      auto bring = [&](int bh, int qt, int kt, int kv_len) {
        const int kvh = kv_head(mk, bh);
        for (int half = 0; half < 2; ++half, ++it) {
          const int s = it % L::kStages;
          if (half == 0 ? !hand_on(bh, qt, kt, kv_len)
                        : !mbar_wait(empty[s], ((it / L::kStages) & 1u) ^ 1u, tmo, abort_flag)) {
            ok = false;
            break;
          }
          mbar_expect_tx(full[s], 2 * T);
          for (int c = 0; c < L::kChunks; ++c) {
            tma_load_3d(sRing + (2 * s) * T + c * 16384, half ? &tm_do : &tm_q, c * 64, qt * kTile,
                        bh, full[s]);
            tma_load_3d(sRing + (2 * s + 1) * T + c * 16384, half ? &tm_v : &tm_k, c * 64,
                        kt * kTile, kvh, full[s]);
          }
        }
      };
      if constexpr (ROWS) {
        const int units = mk.B * mk.H * list.n_q;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
          const int bh = u / list.n_q, qt = u - bh * list.n_q, kv_len = kv_len_of(mk, bh / mk.H);
          const TileRun seen =
              seen_key_tiles(mk, tile_pos(mk, qt), (kv_len + kTile - 1) / kTile);
          if (seen.hi - seen.lo == 1) bring(bh, qt, seen.lo, kv_len);
        }
      } else {
        for (; w.left > 0 && ok; w.next()) {
          group = w.group();
          const int kv_len = kv_len_of(mk, w.b), qt = w.qt(), kt = w.kt();
          if (tile_valid<kRel>(mk, qt, kt, list.n_q, (kv_len + kTile - 1) / kTile))
            bring(w.b * mk.H + w.h, qt, kt, kv_len);
        }
      }
      if (!ok || !hand_on(-1, 0, 0, 0)) fail();
      // every load issued here must land before the CTA exits
      for (int s = 0; s < L::kStages; ++s)
        if (it > static_cast<uint32_t>(s))
          mbar_wait(full[s], ((it - 1 - s) / L::kStages) & 1, tmo, nullptr);
    }
    __syncwarp();
  } else if (warp == kNearMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t kId = idesc_bf16_f32(128, 128, 0, 0);
      uint32_t it = 0;
      bool ok = true;
      while (ok) {
        const uint32_t n = it >> 1, x = n & 1u;  // pairs so far; S and dP buffer
        if (!mbar_wait(pair_full[n % kPairSlots], (n / kPairSlots) & 1u, tmo, abort_flag)) {
          ok = false;
          break;
        }
        if (pairs[2 * (n % kPairSlots)].x < 0) break;
        if (n >= 2 && !mbar_wait(s_free[x], ((n >> 1) - 1) & 1u, tmo, abort_flag)) {
          ok = false;
          break;
        }
        for (uint32_t half = 0; half < 2; ++half, ++it) {
          const int s = it % L::kStages;
          if (!mbar_wait(full[s], (it / L::kStages) & 1u, tmo, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = sdesc_sw128(sRing + (2 * s) * T, 16, 1024);
          const uint64_t db = sdesc_sw128(sRing + (2 * s + 1) * T, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
            mma_ss(tmem + 256u * x + 128u * half, da + off, db + off, kId, kk > 0 ? 1u : 0u);
          }
          mma_commit(empty[s]);
        }
        if (ok) mma_commit(s_full[x]);
      }
      if (!ok) fail();
      mma_commit(drain);
      mbar_wait(drain, 0, tmo, nullptr);
    }
    __syncwarp();
  } else {
    // Warpgroup wg owns key columns [32 wg, 32 wg + 32) of every tile; the thread owns a query row.
    const int wg = warp >> 2, quad = warp & 3;
    const int t = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    float* diag = reinterpret_cast<float*>(smem + L::kDiagOff) + (wg & 1) * kTile * kDiagPitch;
    float* line_s = reinterpret_cast<float*>(smem + L::kLineOff);
    const float c_log2 = args.b.scale_log2;
    const uint64_t c2 = f2_pack(c_log2, c_log2);
    const uint64_t ks2 = f2_pack(args.b.drop.keep_scale, args.b.drop.keep_scale);
    // Barriers with a limit, as every wait here (a warp that gave up does not come to them).
    bool ok = true;
    uint32_t n_all = 0, n_wg = 0;
    auto meet_at = [&](uint32_t bar, uint32_t n) {
      mbar_arrive(bar);
      if (!mbar_wait_warp(bar, n & 1u, tmo, abort_flag)) {
        fail();
        ok = false;
      }
    };
    auto sync_wg = [&]() { meet_at(meet[1 + wg], n_wg++); };
    auto sync_all = [&]() { meet_at(meet[0], n_all++); };
    float acc[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) acc[c] = 0.f;
    // Sums of the accumulated tile along its diagonals, per warpgroup: entry e is the sum of the
    // elements with key column - query row = 32 wg + e - 127. Two warpgroups at a time.
    auto flush = [&](int group) {
      float* out = args.diag_sums +
                   (static_cast<size_t>(group) + blockIdx.x) * kRelDiagFloats + wg * 160;
#pragma unroll
      for (int round = 0; round < 2; ++round) {
        if ((wg >> 1) == round) {
#pragma unroll
          for (int c = 0; c < 32; ++c) diag[t * kDiagPitch + c] = acc[c];
          sync_wg();
          for (int e = t; e < 159; e += 128) {
            // elements (c + 127 - e, c); four sums, so that the loads do not wait for one another
            const int lo = max(0, e - 127), hi = min(31, e);
            const float* at = diag + (127 - e) * kDiagPitch;
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= lo && c <= hi) y[c & 3] += at[c * (kDiagPitch + 1)];
            const float x = (y[0] + y[1]) + (y[2] + y[3]);
            out[e] = x;
          }
        }
        sync_all();
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) acc[c] = 0.f;
    };
    const size_t rows = static_cast<size_t>(mk.B) * mk.H * N;
    int4 p = make_int4(-1, 0, 0, -1), p_next;  // the pair, and the one after it
    int kv_len = 0, kv_next = 0;
    float lse_next = 0.f, d_next = 0.f, r_next[4];  // lse, D and dS sums of the next pair's row
    auto look_ahead = [&](uint32_t n) {
      const uint32_t slot = n % kPairSlots;
      if (!mbar_wait_warp(pair_full[slot], (n / kPairSlots) & 1u, tmo, abort_flag)) {
        fail();
        ok = false;
        return;
      }
      p_next = pairs[2 * slot];
      kv_next = pairs[2 * slot + 1].x;
      const int row = p_next.y * kTile + t;
      lse_next = -INFINITY;
      d_next = r_next[0] = r_next[1] = r_next[2] = r_next[3] = 0.f;
      if (p_next.x >= 0 && row < N) {
        const size_t i = static_cast<size_t>(p_next.x) * N + row;
        lse_next = args.b.lse[i];
        if constexpr (!ROWS) {  // the D of the unrounded O is D and the row's sum of dS
          const float* p = args.b.row_sums + i;
          d_next = args.b.dsum[i];
#pragma unroll
          for (int w = 0; w < 4; ++w) r_next[w] = p[w * rows];
        }
      }
    };
    look_ahead(0);
    const int first_group = ok ? pairs[1].y : -1;
    // the sums of the groups that this CTA's pairs begin and end with, and of those between, are
    // written once each, be there valid pairs or none
    int group = first_group, line_group = -1;
    for (uint32_t n = 0; ok; ++n) {
      p = p_next;
      kv_len = kv_next;
      if (p.w != group) {
        // (the sums of a group without a valid pair here are zeros)
        if (group >= 0)
          for (; group < p.w; ++group) flush(group);
        group = p.w;
        line_group = -1;
      }
      if (p.x < 0) break;
      const int kt = p.z, row = p.y * kTile + t;
      auto tile_distance = [&]() { return kt * kTile - tile_pos(mk, p.y); };
      const int d0 = ROWS ? tile_distance() : 0;
      if (!ROWS && line_group != group) {
        sync_all();  // the line before it is no longer read
        if (tid < 2 * kTile - 1)
          line_s[tid] =
              __ldg(rel_line(args.b.rel, p.x % mk.H) + (tile_distance() - (kTile - 1) + tid));
        sync_all();
        line_group = group;
      }
      const float nl = lse_next == -INFINITY ? -INFINITY : -lse_next * kLog2e;
      const float nd =  // (ROWS: the sum of P Z dP / (1-p) is D)
          ROWS ? 0.f : -(d_next + ((r_next[0] + r_next[1]) + (r_next[2] + r_next[3])));
      const int bh = p.x;
      look_ahead(n + 1);
      if (!ok) break;
      const uint64_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
      int lo = 0, lim = kTile;
      const bool masked = tile_needs_element_mask<kRel>(mk, p.y, kt, kv_len);
      if (masked) visible_keys(mk, row + mk.q_off, kt, kv_len, lo, lim);
      const uint32_t x = n & 1u;
      if (!mbar_wait_warp(s_full[x], (n >> 1) & 1u, tmo, abort_flag)) {
        fail();
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tS = tmem + lane_base + 256u * x + 32u * wg;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t sr[16], dr[16];
        tmem_ld16(tS + 16 * half, sr);
        tmem_ld16(tS + 128 + 16 * half, dr);
        uint4 k4;
        if constexpr (DROPOUT)
          k4 = dropout_keep16(args.b.drop,
                              static_cast<uint32_t>(bh) * static_cast<uint32_t>(N) +
                                  static_cast<uint32_t>(row),
                              static_cast<uint32_t>(kt * 8 + 2 * wg + half));
        tmem_ld_wait();
        if (half == 1) {
          tc_fence_before();
          mbar_arrive(s_free[x]);
        }
        const int c0 = 32 * wg + 16 * half;
        float own[16];  // ROWS: each tile has other distances, and may lie beyond their range
        if constexpr (ROWS) {
          if (args.b.mode != kRel) {
#pragma unroll
            for (int c = 0; c < 16; ++c) own[c] = 0.f;
          } else {
            const RelParams& r = args.b.rel;
            const float* line = rel_line(r, bh % mk.H);
            if (rel_far(r, d0)) {
              const float b = __ldg(line + (rel_far_left(r, d0) ? -r.left : r.right));
#pragma unroll
              for (int c = 0; c < 16; ++c) own[c] = b;
            } else {
              const float4* w = rel_windows(r, line) + (d0 + c0 - t);
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 b = __ldg(w + c);
                own[c] = b.x;
                own[c + 1] = b.y;
                own[c + 2] = b.z;
                own[c + 3] = b.w;
              }
            }
          }
        }
        const float* lp = ROWS ? own : line_s + (127 + c0 - t);
        if (masked) {
          // (a key behind the length may hold anything in V)
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const bool see = c0 + c >= lo && c0 + c < lim;
            sr[c] = see ? sr[c] : 0xFF800000u;  // -inf
            dr[c] = see ? dr[c] : 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          float x0, x1, a0, a1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), c2,
                           f2_add(f2_pack(lp[c], lp[c + 1]), nl2)),
                    x0, x1);
          if constexpr (DROPOUT) {
            const uint32_t wd = c < 4 ? k4.x : c < 8 ? k4.y : c < 12 ? k4.z : k4.w;
            dr[c] &= prmt(wd, 0u, (8u | (c & 3)) * 0x1111u);
            dr[c + 1] &= prmt(wd, 0u, (8u | ((c + 1) & 3)) * 0x1111u);
          }
          const uint64_t t2 =
              f2_fma(ks2, f2_pack(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])), nd2);
          f2_unpack(f2_fma(f2_pack(ex2_approx(x0), ex2_approx(x1)), t2,
                           f2_pack(acc[16 * half + c], acc[16 * half + c + 1])),
                    a0, a1);
          acc[16 * half + c] = a0;
          acc[16 * half + c + 1] = a1;
        }
      }
      if constexpr (ROWS) {  // the row's sum over its four warpgroups
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          sum[c & 3] += acc[c];
          acc[c] = 0.f;
        }
        // A part is written again for pair n + 4, whose S waits until all have read that of pair
        // n + 2, warpgroup 0 after the sums of pair n + 1.
        float* part = reinterpret_cast<float*>(smem + L::kDiagOff) + (n & 3u) * 4 * kTile;
        part[wg * kTile + t] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        mbar_arrive(summed[n & 3u]);
        if (wg == 0) {
          if (!mbar_wait_warp(summed[n & 3u], (n >> 2) & 1u, tmo, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          if (row < N)
            args.b.dsum[static_cast<size_t>(bh) * N + row] =
                (part[t] + part[kTile + t]) + (part[2 * kTile + t] + part[3 * kTile + t]);
        }
      }
    }
    if (!ROWS && group >= 0 && ok) flush(group);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kNearMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ sums by distance
constexpr int kMaxDiags = 640;
constexpr int kOver = 2 * (kTile - 1);  // a near tile reaches that far past either end

// Four threads per distance, one for each warpgroup's part of the diagonals' sums.
__device__ __forceinline__ void line_sums(const RelGradArgs& a, int ctas, int block, int h) {
  __shared__ long long start[kMaxDiags + 1];  // first pair of each group, within a head
  const NearList l = near_list(a);
  for (int g = threadIdx.x; g <= l.n_diag; g += 256) {
    long long n = 0;
    for (int i = 0; i < g; ++i) n += l.count(i);
    start[g] = n * l.B;
  }
  __syncthreads();
  const long long per_head = start[l.n_diag];
  const long long per = max(1ll, near_per_cta(per_head * a.b.mask.H, ctas));
  const int left = a.b.rel.left, right = a.b.rel.right, off = a.b.mask.q_off;
  const int x = block * 64 + static_cast<int>(threadIdx.x >> 2), k = threadIdx.x & 3;
  const int length = left + right + 1 + 2 * kOver;
  float sum = 0.f;
  if (x < length) {
    const int dist = x - left - kOver;
    const int last = floor_tiles(dist + off + (kTile - 1)) - l.first;  // group that reaches it last
    for (int g = max(last - 1, 0); g <= min(last, l.n_diag - 1); ++g) {
      const int e = dist - ((l.first + g) * kTile - off) + (kTile - 1) - 32 * k;
      if (e < 0 || e >= 159 || start[g + 1] == start[g]) continue;
      const long long p0 = h * per_head + start[g], p1 = h * per_head + start[g + 1] - 1;
      const int c1 = static_cast<int>(p1 / per);
      const float* s = a.diag_sums + (static_cast<size_t>(h) * l.n_diag + g) * kRelDiagFloats +
                       160 * k + e;
#pragma unroll 4
      for (int c = static_cast<int>(p0 / per); c <= c1; ++c)
        sum += s[static_cast<size_t>(c) * kRelDiagFloats];
    }
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  if (x < length && k == 0) a.line_sums[static_cast<size_t>(h) * length + x] = sum;
}

// The far fields' sums and those by distance need nothing of one another: one launch (4 us less
// at B = 16, H = 16, N = 1024 than one each).
__global__ void __launch_bounds__(256)
    rel_sums_kernel(const RelGradArgs a, int ctas, int chunks, int line_blocks) {
  const int block = blockIdx.x, n = line_blocks * a.b.mask.H;
  pdl_wait();
  if (block < n)
    line_sums(a, ctas, block % line_blocks, block / line_blocks);
  else
    rows_sums(a, chunks, block - n);
}

// ------------------------------------------------------------------ table
// A block takes 32 buckets of a head, a lane each; its warps share the distances.
__global__ void __launch_bounds__(256) rel_table_kernel(const RelGradArgs a, int chunks) {
  __shared__ Sum part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  const int n = blockIdx.x * 32 + lane;
  pdl_wait();
  const int left = a.b.rel.left, right = a.b.rel.right;
  const int length = left + right + 1 + 2 * kOver;
  const float* line = a.line_sums + static_cast<size_t>(h) * length;
  Sum sum;
  // 32 distances at a time, a lane each, then one after another for all buckets
  for (int x0 = warp * 32; x0 < length; x0 += 256) {
    const int x = x0 + lane;
    const float v = x < length ? line[x] : 0.f;  // (of the kernel in front: no __ldg)
    const int m = __ldg(a.map + clamp_distance(min(x, length - 1) - left - kOver, left, right) + left);
    if (__any_sync(0xffffffffu, (m & ~31) == (n & ~31))) {
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const float vi = __shfl_sync(0xffffffffu, v, i);
        const int mi = __shfl_sync(0xffffffffu, m, i);
        sum.add(mi == n ? vi : 0.f);
      }
    }
  }
  // the far fields: even warps the left one's batch rows, odd warps the right one's
  const int side = warp & 1;
  Sum far;
  for (int i = (warp >> 1) * 32 + lane; i < a.b.mask.B * chunks; i += 128) {
    const size_t bh = static_cast<size_t>(i / chunks) * a.b.mask.H + h;
    far.add(a.far_sums[(bh * chunks + i % chunks) * 2 + side]);
  }
  far.add_lanes();
  if (__ldg(a.map + (side ? left + right : 0)) == n) sum.add(far);
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && n < a.num_buckets) {
    for (int w = 1; w < 8; ++w) sum.add(part[w][lane]);
    a.dtable[static_cast<size_t>(n) * a.b.mask.H + h] = sum.hi + sum.lo;
  }
}

template <int D, bool DROPOUT, bool ROWS>
cudaError_t launch_near(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tdo, const RelGradArgs& a, int ctas,
                        cudaStream_t stream) {
  auto kern = rel_near_kernel<D, DROPOUT, ROWS>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), NearL<D>::kSmemBytes, 0, ready);
  if (e != cudaSuccess) return e;
  return launch_next(kern, dim3(ctas), kNearThreads, NearL<D>::kSmemBytes, stream, tq, tk, tv, tdo, a);
}

template <bool ROWS>
cudaError_t launch_near_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tdo, const RelGradArgs& a, int d, bool dropout,
                          int ctas, cudaStream_t stream) {
  if (d == 64)
    return dropout ? launch_near<64, true, ROWS>(tq, tk, tv, tdo, a, ctas, stream)
                   : launch_near<64, false, ROWS>(tq, tk, tv, tdo, a, ctas, stream);
  return dropout ? launch_near<128, true, ROWS>(tq, tk, tv, tdo, a, ctas, stream)
                 : launch_near<128, false, ROWS>(tq, tk, tv, tdo, a, ctas, stream);
}

}  // namespace

cudaError_t launch_row_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const BwdArgs& b, int d, bool dropout,
                         int num_sms, cudaStream_t stream) {
  const MaskParams& m = b.mask;
  // causal: rows of a tile from position -127 to 0 on see the first key tile alone
  if (m.seqlens_k == nullptr && m.Nk > kTile && m.wl < 0 && m.wr < 0 && !(m.causal && m.q_off <= 0))
    return cudaSuccess;
  RelGradArgs a = {};
  a.b = b;
  const long long units = static_cast<long long>(m.B) * m.H * ((m.N + kTile - 1) / kTile);
  const int ctas = static_cast<int>(units < num_sms ? units : num_sms);
  return launch_near_d<true>(tq, tk, tv, tdo, a, d, dropout, ctas, stream);
}

cudaError_t launch_rel_lines(const RelLinesArgs& a, cudaStream_t stream) {
  const int stride = RelParams{nullptr, a.left, a.right}.stride();
  rel_lines_kernel<<<dim3((stride + 255) / 256, a.H), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rel_grad(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const RelGradArgs& a, int d, bool dropout,
                            int num_sms, cudaStream_t stream) {
  if (a.n_diag > kMaxDiags) return cudaErrorInvalidValue;
  const MaskParams& m = a.b.mask;
  const int chunks = (m.N + kRelRows - 1) / kRelRows;
  cudaError_t e = cudaSuccess;
  const int ctas = num_sms < kRelMaxCtas ? num_sms : kRelMaxCtas;
  if (a.n_diag > 0)
    e = launch_near_d<false>(tq, tk, tv, tdo, a, d, dropout, ctas, stream);
  if (e != cudaSuccess) return e;
  const int length = a.b.rel.left + a.b.rel.right + 1 + 2 * kOver;
  const int line_blocks = (length + 63) / 64;
  e = launch_next(rel_sums_kernel, dim3((line_blocks + chunks * m.B) * m.H), 256, 0, stream, a, ctas,
                  chunks, line_blocks);
  if (e != cudaSuccess) return e;
  return launch_next(rel_table_kernel, dim3((a.num_buckets + 31) / 32, m.H), 256, 0, stream, a, chunks);
}

}  // namespace fa
