// Internal interface between the C-ABI layer (fa_api.cu) and the bf16 forward and
// backward kernels (and their test hooks); decode and FP8 have their own headers.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"

namespace fa {

struct FwdArgs {
  MaskParams mask;
  DropParams drop;
  SyncParams sync;
  float scale_log2;  // scale * log2(e)
  __nv_bfloat16* o;  // [B, H, N, d]
  float* lse;        // [B, H, N]
  int mode;          // Mode
  RelParams rel;     // kRel
};

struct BwdArgs {
  MaskParams mask;
  DropParams drop;
  SyncParams sync;
  float scale;       // softmax scale (dK and dQ are multiplied by it)
  float scale_log2;  // scale * log2(e)
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  const float* lse;  // [B, H, N], natural log
  float* dsum;       // D = rowsum(dO * O), fp32 [B, H, N] (workspace)
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int mode;          // Mode
  RelParams rel;     // kRel
  // kRel, for the gradient of the bias (null: not wanted): what each of the dQ kernel's four
  // warpgroups saw of a query row, [kRelRowSums][4][B*H*N] fp32
  float* row_sums;
  // kCross, kRel with key lengths: the (K/V head, key tile) pairs within them (bhk * tiles + kt, as
  // many as the first entry says), so that the CTAs of the key-tile kernel get even shares. The
  // preprocess kernel lists them, and zeroes the gradients of whole tiles behind the lengths.
  int32_t* key_tiles;
  // kCross, kRel: the key-tile kernel's units per key tile, each with an even share of the query
  // tiles that see it (dkdv_pieces), and for more than one their dK and dV before scaling, fp32
  // [unit][dK, dV][128][d], which launch_dkdv_merge adds up in order.
  int pieces;
  float* dkdv_part;
};

// Unit u of the key-tile kernel is the list's key tile u, in its PIECES instances piece u % pieces
// of key tile u / pieces.
template <bool PIECES>
__device__ __forceinline__ int key_tile_units(const BwdArgs& a, int tiles) {
  return (a.key_tiles != nullptr ? a.key_tiles[0] : a.mask.B * a.mask.Hkv * tiles) *
         (PIECES ? a.pieces : 1);
}
template <bool PIECES>
__device__ __forceinline__ int key_tile_at(const BwdArgs& a, int u) {
  const int i = PIECES ? u / a.pieces : u;
  return a.key_tiles != nullptr ? a.key_tiles[1 + i] : i;
}
// The query tiles 32 chunk .. 32 chunk + 31 of the g-th query head of unit u that its piece has.
__device__ __forceinline__ uint32_t piece_bits(const BwdArgs& a, int u, int kt, int g, int G,
                                               int n_q, int chunk) {
  const TileRun run = seeing_query_tiles(a.mask, kt, n_q);
  const int n = max(0, run.hi - run.lo), piece = u % a.pieces;
  const long long total = static_cast<long long>(n) * G;
  const int from = static_cast<int>(total * piece / a.pieces) - g * n;
  const int to = static_cast<int>(total * (piece + 1) / a.pieces) - g * n;
  const int lo = run.lo + min(max(from, 0), n) - 32 * chunk;
  const int hi = run.lo + min(max(to, 0), n) - 32 * chunk;
  const uint32_t below_lo = lo <= 0 ? 0u : (lo >= 32 ? ~0u : (1u << lo) - 1u);
  const uint32_t below_hi = hi <= 0 ? 0u : (hi >= 32 ? ~0u : (1u << hi) - 1u);
  return below_hi & ~below_lo;
}

// Few key tiles (a short memory, few K/V heads) leave most SMs without a unit: their units are cut
// into pieces where the longest CTA's steps (query tiles, kUnitSteps per unit, kMergeSteps for the
// merge) become fewer. At most kMaxPieces units. The tiles are counted by the keys' length, not by the
// batch's lengths, which are on the device. (B=7 H=16 H_kv=4, 95 keys, 6763 queries, d=64: 94 us with
// the merge against 367. They are instances of their own, so that the others keep their registers.)
constexpr int kMaxPieces = 304;     // what the workspace has room for
constexpr int kMinCutTiles = 10;    // fewer query tiles of a unit: no cut leaves fewer steps
inline int dkdv_pieces(long long key_tiles, long long query_tiles, int num_sms) {
  constexpr long long kUnitSteps = 3, kMergeSteps = 6;
  auto steps = [&](long long s) {
    return (key_tiles * s + num_sms - 1) / num_sms * ((query_tiles + s - 1) / s + kUnitSteps) +
           (s > 1 ? kMergeSteps : 0);
  };
  int best = 1;
  if (query_tiles < kMinCutTiles) return best;
  for (long long s = 2; s * key_tiles <= kMaxPieces && 2 * s <= query_tiles; ++s)
    if (steps(s) < steps(best)) best = static_cast<int>(s);
  return best;
}
cudaError_t launch_dkdv_merge(const BwdArgs& a, int d, cudaStream_t stream);

// Sums over the keys of a query row: dS, dS left of the range of distances, dS right of it, P
// not left of it, P right of it.
constexpr int kRelRowSums = 5;

// Tensor maps of a [B*H, N, d] bf16 tensor with 128 x 64 boxes, 128-byte swizzle.
cudaError_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const FwdArgs& a, int d, bool dropout, int num_sms, cudaStream_t stream);

// d = 128 forward (fa_fwd128.cu); launch_fwd routes d = 128 there.
cudaError_t launch_fwd128(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const FwdArgs& a, bool dropout, int num_sms, cudaStream_t stream);

cudaError_t launch_bwd_preprocess(const BwdArgs& a, int d, int num_sms, cudaStream_t stream);

cudaError_t launch_bwd_dkdv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const BwdArgs& a, int d, bool dropout,
                            int num_sms, cudaStream_t stream);

cudaError_t launch_bwd_dq(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tdo, const BwdArgs& a, int d, bool dropout,
                          int num_sms, cudaStream_t stream);

// Two-issuer backward kernels (fa_bwd_split.cu): dK/dV at d = 64 (d = 128 runs the
// single-issuer kernel of fa_bwd.cu), dQ at d = 64 or 128.
cudaError_t launch_bwd_dkdv_split(const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const CUtensorMap& tdo, const BwdArgs& a,
                                  int d, bool dropout, int num_sms, cudaStream_t stream);
cudaError_t launch_bwd_dq_split(const CUtensorMap& tq, const CUtensorMap& tk,
                                const CUtensorMap& tv, const CUtensorMap& tdo, const BwdArgs& a,
                                int d, bool dropout, int num_sms, cudaStream_t stream);

// Relative position bias (fa_rel.cu).
struct RelLinesArgs {
  const void* table;   // [num_buckets, H], fp32 or bf16
  bool bf16;
  const int32_t* map;  // [left + right + 1]
  int left, right, num_buckets, H;
  float* lines;
  unsigned int* status;
};
cudaError_t launch_rel_lines(const RelLinesArgs& a, cudaStream_t stream);

struct RelGradArgs {
  BwdArgs b;             // with the dQ kernel's row_sums
  const int32_t* map;
  int num_buckets;
  float* dtable;         // [num_buckets, H]
  int first, n_diag;     // near tile pairs: kt - qt = first .. first + n_diag - 1
  float* diag_sums;      // [H * n_diag + kRelMaxCtas][4][160]
  float* line_sums;      // [H, left + right + 1 + 508], by distance from -left - 254 on
  float* far_sums;       // [B * H, ceil(N / kRelRows)][2]
};
constexpr int kRelMaxCtas = 512;
constexpr int kRelRows = 256;       // query rows whose far sums a block forms
constexpr int kRelDiagFloats = 640; // 4 warpgroups x 160 diagonals
cudaError_t launch_rel_grad(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const RelGradArgs& a, int d, bool dropout,
                            int num_sms, cudaStream_t stream);

// kCross, kRel: D of the query tiles whose rows see one key tile, from their scores (nothing is
// launched where there can be none). After launch_bwd_preprocess, whose D it replaces.
cudaError_t launch_row_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const BwdArgs& a, int d, bool dropout,
                         int num_sms, cudaStream_t stream);

cudaError_t launch_debug_dropout(uint8_t* keep, int B, int H, int N, const DropParams& d,
                                 cudaStream_t stream);

cudaError_t launch_debug_philox(const uint32_t* counters, uint32_t* out, int n, uint32_t k0,
                                uint32_t k1, cudaStream_t stream);

}  // namespace fa
