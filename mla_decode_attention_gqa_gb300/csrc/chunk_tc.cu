// Tensor-core (tcgen05) attention of ragged chunks of new tokens over a paged cache
// (attn_chunk_paged): prompt chunks, proposed tokens and decode tokens of one packed batch,
// causal or with a sliding window and sinks; bf16 pages.
//
// For every row (new token at position p, query head h of KV head g): s_u = scale q.k_u over
// the visible tokens u (u <= p and u > p - window or u < n_sink), out = softmax(s) V, lse =
// ln sum e^s.  One pass over the tokens with a running maximum; sums and O in fp32, P rounded
// to bf16 for the product with V (2^-8 of each weight at most, as much as the output's own
// rounding).  O is divided by the fp32 sum of the unrounded weights: summing the rounded ones as
// well cost two more additions a pair of scores on the path that bounds the kernel.
//
// Bound by the tensor pipe for chunks of 128 and more rows (two 128 x 128 x D products per tile
// of 128 tokens and 128 rows), by HBM for few rows.  Design (one CTA an SM, 384 threads):
//   * rows of one KV head are (token, head of the group) pairs, the group padded to a power of
//     two Gr, so that a 128-row tile is a TMA box of 128 / Gr tokens x Gr heads; every K/V byte
//     is read once for the whole group;
//   * warps 0 and 2 load (Q once; K and V tiles of 128 tokens, each 64-token half from its own
//     page, into separate K and V rings, since a K tile is free as soon as its scores are done
//     and a V tile only after the softmax), warp 1 issues every MMA, warps 4-7 and 8-11 are two
//     softmax groups with one thread a row (the TMEM lane of its row: no shuffles);
//   * pair mode (an item of more than 128 rows): group k serves query tile k, both read each
//     K/V tile; MMA order PV0(i), S0(i+1), PV1(i), S1(i+1), so that one group works while the
//     tensor pipe serves the other;
//   * solo mode (128 rows or fewer, a decode token's group say): both groups serve the one query
//     tile on alternate K/V tiles with an O each, joined in the epilogue: the chain load, S,
//     softmax, PV of one tile is latency, and two run side by side.  Warps without a row skip
//     the softmax;
//   * TMEM: S0 | S1 | O0 | O1; P in bf16 over its S, read from TMEM as the A operand of P V.
//     MMAs from one thread complete in order, so when S_k(i+1) has landed PV_k(i) is done and
//     O_k may be rescaled;
//   * optimistic softmax: p = 2^(s - m) against the maximum so far; only a row's first visible
//     tile, and a tile whose p sum passes 2^16, take the tile's maximum, rescale O and redo.
#include <climits>
#include <cuda_runtime.h>

#include <type_traits>

#include "chunk_plan.cuh"
#include "skv_common.cuh"
#include "skv_internal.h"
#include "tc_common.cuh"

namespace skv {

namespace {

constexpr int kTN = 128;        // tokens per K/V tile
constexpr int kHalf = kTN / 2;  // tokens per TMA box: a page holds a multiple of 64
constexpr int kRowsTile = 128;  // rows per query tile (MMA M)
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S_k (P_k over its first 64 columns) at kColS + 128 k
constexpr uint32_t kColO = 256;  // O_k at kColO + 128 k
constexpr float kTileSumLimit = 65536.0f;

template <int D_>
struct TcCfg {
  static constexpr int D = D_;
  static constexpr int NB = D / 64;                  // 128-byte boxes of a row
  static constexpr int NST = D == 64 ? 4 : 2;        // ring depth, tiles
  static constexpr int BOX = kTN * 128;              // one box column of a tile: 128 rows x 128 bytes
  static constexpr int TILE = NB * BOX;              // a Q, K or V tile of 128 rows
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NST * TILE;
  static constexpr int OFF_BAR = OFF_V + NST * TILE;
  static constexpr int OFF_ML = OFF_BAR + 256;       // solo: group 1's (m, l) per row
  static constexpr int SMEM = 1024 + OFF_ML + kRowsTile * 8;
  static_assert(SMEM <= 226 * 1024, "shared memory budget (the work search has some of its own)");
};

template <class C>
struct TcBars {
  uint64_t q_full;
  uint64_t k_full[C::NST], k_empty[C::NST];
  uint64_t v_full[C::NST], v_empty[C::NST];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint32_t tmem_base;
};

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

template <int V>
using Int = std::integral_constant<int, V>;

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ PartialParams p, const __grid_constant__ CUtensorMap tmq,
                    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  constexpr int D = C::D, NST = C::NST, NB = C::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBars<C>* bars = reinterpret_cast<TcBars<C>*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  ChunkItem it;
  if (!chunk_find_item<kThreads>(p.ck, &it)) return;
  const int G = p.ck.G, Gr = p.ck.group_rows;
  const int rows_total = it.n * Gr;
  const int m0 = it.mt * 2 * kRowsTile;
  const int m_last = min(m0 + 2 * kRowsTile, rows_total) - 1;
  const bool pair = m_last - m0 >= kRowsTile;
  const int pos0 = it.m - it.n;  // position of the sequence's first row
  const ChunkTiles tl = chunk_tiles(p.ck.window, p.ck.n_sink, p.ck.cap, pos0 + m0 / Gr, pos0 + m_last / Gr, kTN);
  const int per_chunk = (tl.n + it.n_chunk - 1) / it.n_chunk;
  const int i0 = min(it.c * per_chunk, tl.n);
  const int n_tiles = min(per_chunk, tl.n - i0);
  auto tile_token = [&](int i) -> int {  // first token of the chunk's tile i
    const int x = i0 + i;
    return (x < tl.n_first ? x : tl.win + (x - tl.n_first)) * kTN;
  };

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&bars->s_full[k], 1);
      mbar_init(&bars->p_full[k], kRowsTile);
      mbar_init(&bars->pv_done[k], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers: 0 Q and K, 2 V
    // A warp each, so that neither waits for the other's ring; the pages and rows of the next
    // tile (four integer divisions and two dependent loads) are looked up behind this tile's
    // copies, not between a freed stage and its refill, which bounds a two-stage ring.
    if (n_tiles > 0) {
      const bool is_k = warp == 0;
      const CUtensorMap* map = is_k ? &tmk : &tmv;
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      uint8_t* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
      if (tc::elect_one()) {
        tma_prefetch_desc(map);
        if (is_k) {
          tma_prefetch_desc(&tmq);
          const int nq = pair ? 2 : 1;
          mbar_arrive_expect_tx(&bars->q_full, nq * C::TILE);
          for (int k = 0; k < nq; ++k)
            for (int bx = 0; bx < NB; ++bx)
              tma_4d(smem + k * C::TILE + bx * C::BOX, &tmq, &bars->q_full, bx * 64, it.g * G,
                     it.row0 + (m0 + k * kRowsTile) / Gr, 0);
        }
      }
      __syncwarp();
      int page[2], at[2];  // of a tile's two halves
      auto look_up = [&](int i) {
        const int t = tile_token(i);
        // a second half at or past the capacity holds no token: it takes the first one's page
        // instead of an entry behind the table's row
        const int t2 = t + kHalf < p.ck.cap ? t + kHalf : t;
        at[0] = t % p.block_len;
        at[1] = t2 % p.block_len;
        page[0] = kv_page_of(p, it.b, t);
        page[1] = kv_page_of(p, it.b, t2);
      };
      look_up(0);
      int issued = 0;
      for (int i = 0; i < n_tiles; ++i) {
        const int s = i % NST;
        if (i >= NST && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((i / NST) - 1) & 1, p.err, kDevErrEmptyWait))) break;
        if (tc::elect_one()) {
          mbar_arrive_expect_tx(&full[s], C::TILE);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int bx = 0; bx < NB; ++bx)
              tma_4d(ring + s * C::TILE + bx * C::BOX + hf * (C::BOX / 2), map, &full[s], bx * 64, at[hf], it.g, page[hf]);
        }
        __syncwarp();
        issued = i + 1;
        if (issued < n_tiles) look_up(issued);
      }
      // every issued copy lands before the CTA may exit
      for (int i = max(0, issued - NST); i < issued; ++i)
        if (!mbar_wait(&full[i % NST], (i / NST) & 1, p.err, kDevErrDrainWait)) break;
      if (is_k) mbar_wait(&bars->q_full, 0, p.err, kDevErrDrainWait);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp waits, one elected lane issues; stages are compile-time constants (the
    // loops are unrolled by the ring depth), so every operand is a constant offset.
    if (n_tiles > 0) {
      const uint32_t idesc_s = tc::idesc_f16(128, kTN, true, false, false);
      const uint32_t idesc_pv = tc::idesc_f16(128, D, true, false, true);
      const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
      const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), C::BOX, 1024);
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err, kDevErrFullWait));
      };
      auto issue_s = [&](int k, int q, int stage) {  // S_k = Q_q K^T
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t in_box = (ks >> 2) * C::BOX + (ks & 3) * 32;
          tc::mma_f16_ss(tmem + kColS + 128 * k, qd + static_cast<uint64_t>((q * C::TILE + in_box) >> 4),
                         kd + static_cast<uint64_t>((stage * C::TILE + in_box) >> 4), idesc_s, ks > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int k, int stage, uint32_t acc0) {  // O_k += P_k V
#pragma unroll
        for (int ks = 0; ks < kTN / 16; ++ks)
          tc::mma_f16_ts(tmem + kColO + 128 * k, tmem + kColS + 128 * k + ks * 8,
                         vd + static_cast<uint64_t>((stage * C::TILE + ks * 2048) >> 4), idesc_pv, ks > 0 ? 1u : acc0);
      };
      bool ok = wait_all(&bars->q_full, 0);
      if (pair) {
        // tile i in stage ST: PV0(i), S0(i+1), PV1(i), S1(i+1)
        auto tile = [&](auto st, int i) {
          constexpr int ST = decltype(st)::value, NX = (ST + 1) % NST;
          ok = wait_all(&bars->p_full[0], i & 1) && wait_all(&bars->v_full[ST], (i / NST) & 1);
          if (!ok) return;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_pv(0, ST, i > 0 ? 1u : 0u);
            tc::mma_commit(smem_u32(&bars->pv_done[0]));
          }
          __syncwarp();
          const bool more = i + 1 < n_tiles;
          if (more) {
            ok = wait_all(&bars->k_full[NX], ((i + 1) / NST) & 1);
            if (!ok) return;
            tc::fence_after_sync();
            if (tc::elect_one()) {
              issue_s(0, 0, NX);
              tc::mma_commit(smem_u32(&bars->s_full[0]));
            }
            __syncwarp();
          }
          ok = wait_all(&bars->p_full[1], i & 1);
          if (!ok) return;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_pv(1, ST, i > 0 ? 1u : 0u);
            tc::mma_commit(smem_u32(&bars->pv_done[1]));
            tc::mma_commit(smem_u32(&bars->v_empty[ST]));
            if (more) {
              issue_s(1, 1, NX);
              tc::mma_commit(smem_u32(&bars->s_full[1]));
              tc::mma_commit(smem_u32(&bars->k_empty[NX]));
            }
          }
          __syncwarp();
        };
        ok = ok && wait_all(&bars->k_full[0], 0);
        if (ok) {
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_s(0, 0, 0);
            tc::mma_commit(smem_u32(&bars->s_full[0]));
            issue_s(1, 1, 0);
            tc::mma_commit(smem_u32(&bars->s_full[1]));
            tc::mma_commit(smem_u32(&bars->k_empty[0]));
          }
          __syncwarp();
        }
        for (int i = 0; i < n_tiles && ok; i += NST) {
          tile(Int<0>{}, i);
          if (ok && i + 1 < n_tiles) tile(Int<1>{}, i + 1);
          if constexpr (NST == 4) {
            if (ok && i + 2 < n_tiles) tile(Int<2>{}, i + 2);
            if (ok && i + 3 < n_tiles) tile(Int<3>{}, i + 3);
          }
        }
      } else {
        // tile i in stage ST belongs to group i & 1: PV(i), then S(i + 2)
        auto scores = [&](auto st, int i) {
          constexpr int ST = decltype(st)::value;
          ok = wait_all(&bars->k_full[ST], (i / NST) & 1);
          if (!ok) return;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_s(ST & 1, 0, ST);
            tc::mma_commit(smem_u32(&bars->s_full[ST & 1]));
            tc::mma_commit(smem_u32(&bars->k_empty[ST]));
          }
          __syncwarp();
        };
        auto tile = [&](auto st, int i) {
          constexpr int ST = decltype(st)::value, K = ST & 1;
          ok = wait_all(&bars->p_full[K], (i >> 1) & 1) && wait_all(&bars->v_full[ST], (i / NST) & 1);
          if (!ok) return;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_pv(K, ST, i > 1 ? 1u : 0u);
            tc::mma_commit(smem_u32(&bars->pv_done[K]));
            tc::mma_commit(smem_u32(&bars->v_empty[ST]));
          }
          __syncwarp();
          if (i + 2 < n_tiles) scores(Int<(ST + 2) % NST>{}, i + 2);
        };
        if (ok) scores(Int<0>{}, 0);
        if (ok && n_tiles > 1) scores(Int<1>{}, 1);
        for (int i = 0; i < n_tiles && ok; i += NST) {
          tile(Int<0>{}, i);
          if (ok && i + 1 < n_tiles) tile(Int<1>{}, i + 1);
          if constexpr (NST == 4) {
            if (ok && i + 2 < n_tiles) tile(Int<2>{}, i + 2);
            if (ok && i + 3 < n_tiles) tile(Int<3>{}, i + 3);
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax groups
    const int k = (warp - 4) >> 2;
    const int lgrp = warp & 3;         // TMEM lane group of this warp
    const int row = lgrp * 32 + lane;  // row inside the query tile
    const int m = m0 + (pair ? k * kRowsTile : 0) + row;
    const int t_q = m / Gr, hg = m % Gr;
    const bool valid = m < rows_total && hg < G;
    const int pos = pos0 + t_q;
    // visible tokens of this row: [lo_row, hi_row) and [0, sink_row)
    const int hi_row = valid ? min(max(pos + 1, 0), p.ck.cap) : 0;
    const int lo_row = (valid && p.ck.window > 0 && pos >= p.ck.window) ? pos - p.ck.window + 1 : 0;
    const int sink_row = min(p.ck.n_sink, hi_row);
    const bool active = __any_sync(0xffffffffu, valid);  // some row of this warp exists
    const int hi_min = __reduce_min_sync(0xffffffffu, valid ? hi_row : INT_MAX);
    const int hi_max = __reduce_max_sync(0xffffffffu, hi_row);
    const int lo_max = __reduce_max_sync(0xffffffffu, lo_row);
    const int sink_min = __reduce_min_sync(0xffffffffu, valid ? sink_row : INT_MAX);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lgrp * 32) << 16);
    const uint32_t s_col = t_lane + kColS + 128 * k;
    const uint32_t o_col = t_lane + kColO + 128 * k;
    const float sl = p.scale_log2;
    float m_used = -INFINITY, l_sum = 0.f;
    bool ok = true;
    const int first = pair ? 0 : k, step = pair ? 1 : 2;  // this group's tiles

    int j = 0;  // tiles done
    for (int i = first; i < n_tiles; i += step, ++j) {
      const int t0 = tile_token(i);
      ok = mbar_wait(&bars->s_full[k], j & 1, p.err, kDevErrFullWait);
      if (!ok) break;
      tc::fence_after_sync();
      if (active) {
        const bool none = hi_max <= t0;  // no row of the warp reaches this tile
        const bool need_mask = hi_min < t0 + kTN || (t0 < lo_max && t0 + kTN > sink_min);
        const int c_lo = min(max(lo_row - t0, 0), kTN);
        const unsigned span = static_cast<unsigned>(max(min(max(hi_row - t0, 0), kTN) - c_lo, 0));
        const int c_sink = min(max(sink_row - t0, 0), kTN);
        auto visible = [&](int col) -> bool { return static_cast<unsigned>(col - c_lo) < span || col < c_sink; };
        uint32_t pk[kTN / 2];
        uint64_t ls[2] = {0ull, 0ull};  // fp32 pair sums of p
        const float base0 = (m_used == -INFINITY) ? 0.f : m_used;
        // masked: a compile-time flag, so that tiles that every row sees carry no test
        auto pass = [&](auto masked) {
#pragma unroll
          for (int cc = 0; cc < kTN / 32; ++cc) {
            uint32_t r[2][16];
            tc::tmem_ld16(s_col + 32 * cc, r[0]);
            tc::tmem_ld16(s_col + 32 * cc + 16, r[1]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int col = 32 * cc + 2 * e;
              float v0 = __uint_as_float(r[e >> 3][(2 * e) & 15]);
              float v1 = __uint_as_float(r[e >> 3][(2 * e + 1) & 15]);
              if constexpr (decltype(masked)::value) {
                v0 = visible(col) ? v0 : -INFINITY;
                v1 = visible(col + 1) ? v1 : -INFINITY;
              }
              float a0, a1;
              fma_pair(v0, v1, sl, -base0, a0, a1);
              const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
              ls[e & 1] = add_f32x2(ls[e & 1], p0, p1);
              pk[16 * cc + e] = pack_bf16(p0, p1);
            }
          }
        };
        if (none) {
#pragma unroll
          for (int e = 0; e < kTN / 2; ++e) pk[e] = 0u;
        } else if (need_mask) {
          pass(std::true_type{});
        } else {
          pass(std::false_type{});
        }
        const float tile_sum = sum_f32x2(ls[0]) + sum_f32x2(ls[1]);
        const bool row_vis = valid && !none && (!need_mask || span > 0u || c_sink > 0);
        const bool need = row_vis && (m_used == -INFINITY || !(tile_sum <= kTileSumLimit));
        if (__any_sync(0xffffffffu, need)) {
          // the tile's true maximum, O and l rescaled to it, and this tile's P again from S
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int cc = 0; cc < kTN / 32; ++cc) {
            uint32_t r[2][16];
            tc::tmem_ld16(s_col + 32 * cc, r[0]);
            tc::tmem_ld16(s_col + 32 * cc + 16, r[1]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int col = 32 * cc + 2 * e;
              const float v0 = visible(col) ? __uint_as_float(r[e >> 3][(2 * e) & 15]) : -INFINITY;
              const float v1 = visible(col + 1) ? __uint_as_float(r[e >> 3][(2 * e + 1) & 15]) : -INFINITY;
              mx[e & 3] = fmax3(mx[e & 3], v0, v1);
            }
          }
          const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;  // sl > 0
          const float m_new = need ? fmaxf(m_used, tmax) : m_used;
          if (j > 0) {
            // PV_k of this group's tile before ran before these scores: O_k is final here
            const float alpha = need ? fast_exp2(m_used - ((m_new == -INFINITY) ? 0.f : m_new)) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t r[2][16];
              tc::tmem_ld16(o_col + 16 * c, r[0]);
              tc::tmem_ld16(o_col + 16 * (c + 1), r[1]);
              tc::tmem_wait_ld();
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int e = 0; e < 16; ++e) r[h2][e] = __float_as_uint(__uint_as_float(r[h2][e]) * alpha);
              tc::tmem_st16(o_col + 16 * c, r[0]);
              tc::tmem_st16(o_col + 16 * (c + 1), r[1]);
            }
            tc::tmem_wait_st();
            l_sum *= alpha;
          }
          m_used = m_new;
          const float base = (m_used == -INFINITY) ? 0.f : m_used;
          ls[0] = ls[1] = 0ull;
#pragma unroll 1
          for (int cc = 0; cc < kTN / 32; ++cc) {
            uint32_t r[2][16];
            tc::tmem_ld16(s_col + 32 * cc, r[0]);
            tc::tmem_ld16(s_col + 32 * cc + 16, r[1]);
            tc::tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int col = 32 * cc + 2 * e;
              const float v0 = visible(col) ? __uint_as_float(r[e >> 3][(2 * e) & 15]) : -INFINITY;
              const float v1 = visible(col + 1) ? __uint_as_float(r[e >> 3][(2 * e + 1) & 15]) : -INFINITY;
              const float p0 = fast_exp2(fmaf(v0, sl, -base)), p1 = fast_exp2(fmaf(v1, sl, -base));
              ls[e & 1] = add_f32x2(ls[e & 1], p0, p1);
              w[e] = pack_bf16(p0, p1);
            }
            tc::tmem_st16(s_col + 16 * cc, w);  // S columns 32 cc.. were read before P 16 cc.. is written
          }
        } else {
#pragma unroll
          for (int cc = 0; cc < kTN / 32; ++cc) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pk[16 * cc + e];
            tc::tmem_st16(s_col + 16 * cc, w);
          }
        }
        tc::tmem_wait_st();
        l_sum += sum_f32x2(ls[0]) + sum_f32x2(ls[1]);
      }
      const bool inside = (t0 >= tl.lo && t0 + kTN <= tl.hi) || t0 + kTN <= tl.sinks;
      if (!inside && (k == 0 || !pair)) {
        // tokens that no row of the item sees may hold anything: zero their V rows, so that p = 0
        // really counts nothing
        const int s = i % NST;
        mbar_wait(&bars->v_full[s], (i / NST) & 1, p.err, kDevErrFullWait);
        const int tok = t0 + row;
        if (!((tok >= tl.lo && tok < tl.hi) || tok < tl.sinks)) {
          uint8_t* vt = smem + C::OFF_V + s * C::TILE + row * 128;
          for (int bx = 0; bx < NB; ++bx)
            for (int cc = 0; cc < 8; ++cc)
              *reinterpret_cast<uint4*>(vt + bx * C::BOX + cc * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc::fence_before_sync();
      mbar_arrive(&bars->p_full[k]);
    }

    // ---- epilogue: O / l and lse
    auto tiles_of = [&](int kk) { return pair ? n_tiles : (n_tiles + 1 - kk) / 2; };
    float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
    // solo: the two groups' weights.  A group that summed nothing has l = 0 (its O may be
    // anything); a NaN among the scores keeps l NaN, and the row is NaN
    float a0 = 1.f, a1 = 0.f;
    bool some0 = l_sum != 0.f, some1 = false;
    if (!pair) {
      if (k == 1) {
        ml[2 * row] = m_used;
        ml[2 * row + 1] = l_sum;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (k == 0) {
        const float m1 = ml[2 * row], l1 = ml[2 * row + 1];
        const float mm = fmaxf(m_used, m1);
        some1 = l1 != 0.f;
        a0 = some0 ? fast_exp2(m_used - mm) : 0.f;
        a1 = some1 ? fast_exp2(m1 - mm) : 0.f;
        l_sum = (some0 ? a0 * l_sum : 0.f) + (some1 ? a1 * l1 : 0.f);
        m_used = mm;
      }
    }
    if (pair || k == 0) {
      if (ok && tiles_of(k) > 0) ok = mbar_wait(&bars->pv_done[k], (tiles_of(k) - 1) & 1, p.err, kDevErrFullWait);
      const bool both = !pair && tiles_of(1) > 0;
      if (ok && both) ok = mbar_wait(&bars->pv_done[1], (tiles_of(1) - 1) & 1, p.err, kDevErrFullWait);
      tc::fence_after_sync();
      const bool some = some0 || some1;
      const float inv = some ? 1.f / l_sum : 0.f;
      a0 *= inv;
      a1 *= inv;
      constexpr float kLn2 = 0.6931471805599453f;
      const float lse = some ? (m_used + __log2f(l_sum)) * kLn2 : -INFINITY;
      const bool direct = it.n_chunk == 1;
      const int h = it.g * G + hg;
      const int64_t orow = direct ? (static_cast<int64_t>(it.row0) + t_q) * p.Hq + h
                                  : it.part_row + (static_cast<int64_t>(it.c) * it.n + t_q) * p.Hq + h;
      // an empty partial's o is never read
      const bool write_o = valid && (direct || some);
      if (active) {
#pragma unroll 2
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r[16], r1[16];
          if (n_tiles > 0) tc::tmem_ld16(o_col + 16 * c, r);
          if (both) tc::tmem_ld16(o_col + 128 + 16 * c, r1);
          tc::tmem_wait_ld();
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = some0 ? __uint_as_float(r[e]) * a0 : 0.f;
            if (some1) x[e] = fmaf(__uint_as_float(r1[e]), a1, x[e]);
          }
          if (write_o) {
            if (direct) {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.ck.out) + orow * D + 16 * c;
              *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                        pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
              *reinterpret_cast<uint4*>(o + 8) = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]),
                                                            pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
            } else {
              float* o = p.out_o + orow * D + 16 * c;
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(o + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
          }
        }
      }
      if (valid) (direct ? p.ck.lse : p.out_lse)[orow] = lse;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
}

template <class C>
cudaError_t launch_cfg(const PartialParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                       int64_t n_items, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e0 = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(chunk_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e0 != cudaSuccess) return e0;
  if (n_items <= 0) return cudaSuccess;
  chunk_tc_kernel<C><<<static_cast<unsigned int>(n_items), kThreads, C::SMEM, stream>>>(p, tmq, tmk, tmv);
  return cudaGetLastError();
}

}  // namespace

int chunk_tc_rows() { return 2 * kRowsTile; }
int chunk_tc_kv_tile() { return kTN; }
int chunk_tc_kv_box() { return kHalf; }

cudaError_t launch_chunk_tc(const PartialParams& p, int32_t d, const CUtensorMap& tmq, const CUtensorMap& tmk,
                            const CUtensorMap& tmv, int64_t n_items, cudaStream_t stream) {
  if (d == 64) return launch_cfg<TcCfg<64>>(p, tmq, tmk, tmv, n_items, stream);
  return launch_cfg<TcCfg<128>>(p, tmq, tmk, tmv, n_items, stream);
}

}  // namespace skv
