// Attention of few new tokens over a paged cache (attn_chunk_paged): decode steps and proposed
// tokens, 16 or 32 rows (new token, head of the group) of a KV head at a time, causal or with a
// sliding window and sinks; bf16 pages, fp8-e4m3 pages with block scales, or 4-bit pages (e2m1 codes,
// an e4m3 scale for each 16 dims of a token's head and an fp32 scale a head).
//
// For every row (new token at position p, query head h of KV head g): s_u = scale q.k_u over the
// visible tokens u (u <= p and u > p - window or u < n_sink), out = softmax(s) V, lse = ln sum e^s,
// in one pass with a running maximum; scores, sums and O in fp32.  P is rounded once for the
// product with V: to bf16 (2^-8 of each weight), or times the V block scale to fp16 (2^-11).
//
// Bound by HBM: each K/V byte is read once for the whole group.  A warp loads K and V tiles of 64
// tokens by TMA into a ring; 3 to 5 warps take the tiles in turn (16 x 64 scores on mma.sync
// tiles: tcgen05's 128 rows would be mostly padding) and join their (m, l, O) at the end.  For 17 to
// 32 rows a second set of warps takes the same tiles for the other 16: one CTA an SM with twice the
// ring, where two row tiles would read the pages twice.
//
// Work: the KV tiles of all items (sequence, row tile, KV head) in one line, cut into as many equal
// runs as CTAs are resident: every CTA streams the same number of tiles (an item's start counted as
// some, kChunkStart) and starts once, where chunks of equal length per sequence left a part of a
// wave empty and started four times (decode of 64 sequences of 4096 to 16384 tokens, 64 / 8 heads:
// 404 us, in equal runs 374: the rate of a plain copy).
// A run may begin and end inside an item: those two pieces go out as partial rows, at most
// two a CTA, which chunk_runs_merge joins; the items between are final.
//
// 4-bit pages are bound by the instructions that widen them, at 1.9 a cycle of the 10 warps that 168 registers leave
// (see chunk_rows4.cu, which takes up to 8 rows): decode of 8 sequences of 65536 to 131072 tokens, 128 / 8 heads,
// 223 us, 0.57 of the measured copy rate.  Queries in
// registers for two chunks of 32 dims, four independent products between two into the same scores, both tokens'
// nibbles of V brought into one byte by four operations for 8 codes: 252 -> 234.
#include <cuda_runtime.h>

#include "chunk_plan.cuh"
#include "skv_common.cuh"
#include "skv_internal.h"
#include "warp_wait.cuh"

namespace skv {

namespace {

constexpr int kRows = 16;  // rows of a warp

template <PageFormat PAGES_, int D_, int WM_, int WN_, int NSTAGE_, bool SHARED_>
struct RowsCfg {
  static constexpr PageFormat PAGES = PAGES_;
  static constexpr bool SHARED = SHARED_;  // a pass of a shared prefix (ChunkArgs)
  static constexpr bool FP4 = PAGES == kPagesFp4;
  static constexpr bool FP8 = PAGES == kPagesFp8;
  static constexpr bool CODES = PAGES != kPagesBf16;  // the products run in fp16, P V as V^T P^T
  static constexpr int D = D_;
  static constexpr int WM = WM_;          // sets of 16 rows, which share the tiles
  static constexpr int WN = WN_;          // consumer warps of a set
  static constexpr int ROWS = WM * kRows;
  static constexpr int CTAS = WM == 1 ? 2 : 1;  // an SM
  static constexpr int NSTAGE = NSTAGE_;  // tiles in the ring
  static constexpr int TN = kTileN;
  static constexpr int ESZ = CODES ? 1 : 2;
  static constexpr int NBOX = FP4 ? 1 : D * ESZ / 128;  // 128-byte boxes of a token row (4-bit: one of 64)
  static constexpr int BOX_ELEMS = 128 / ESZ;
  static constexpr int BOX_BYTES = FP4 ? TN * (D / 2) : TN * 128;
  static constexpr int TILE = NBOX * BOX_BYTES;
  static constexpr int SCALES = FP4 ? TN * (D / kFp4Block) : 0;  // 4-bit: the scales of a tile's blocks
  static constexpr int STAGE = 2 * (TILE + SCALES);  // K, V, K's scales, V's
  static constexpr int THREADS = (WM * WN + 1) * 32;
  // Full barriers are per consumer warp (of each set), DW of them each: a warp's wait is then always for the
  // phase after the one it saw last, whatever the other warps' tiles do
  static constexpr int DW = (NSTAGE + WN - 1) / WN;
  static constexpr int NFULL = WN * DW;
  static constexpr int OFF_O = NSTAGE * STAGE;                 // one warp's O of each set, to be joined
  static constexpr int OFF_ML = OFF_O + ROWS * D * 4;          // (m, l) of each warp's rows
  static constexpr int OFF_QF = OFF_ML + WN * ROWS * 2 * 4;    // codes: q fragments
  static constexpr int OFF_BAR = OFF_QF + (CODES ? WM * (D / 16) * 32 * 16 : 0);
  static constexpr int OFF_QS = OFF_BAR + 256;                 // codes: the score scale of each row
  static constexpr int OFF_RUN = OFF_QS + (CODES ? ROWS * 4 : 0);  // each consumer warp's run and piece
  static constexpr int SMEM = 1024 + OFF_RUN + WM * WN * 192;
  static_assert((NFULL + NSTAGE) * 8 <= 256, "barriers");
  static_assert(CTAS * (SMEM + 1536) <= 227 * 1024, "CTAs an SM");
};

template <class C>
__device__ __forceinline__ int full_slot(int x) {  // barrier of tile number x of this CTA
  return (x % C::WN) * C::DW + (x / C::WN) % C::DW;
}
template <class C>
__device__ __forceinline__ uint32_t full_parity(int x) {
  return static_cast<uint32_t>((x / C::WN) / C::DW) & 1u;
}
template <class C>
__device__ __forceinline__ uint32_t tile_off(uint32_t tok, uint32_t byte) {
  return (byte >> 7) * C::BOX_BYTES + swz128(tok, byte & 127u);
}
// Byte `byte` of token `tok`'s row of a 4-bit tile: 64-byte rows under the 64-byte swizzle.
__device__ __forceinline__ uint32_t tile4_off(uint32_t tok, uint32_t byte) {
  return tok * 64u + ((((byte >> 4) ^ ((tok >> 1) & 3u)) << 4) | (byte & 15u));
}
__device__ __forceinline__ uint32_t half_mask(bool lo, bool hi) {
  return (lo ? 0x0000FFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
}
template <class C>
__device__ __forceinline__ void consumers_sync(int set) {  // the consumer warps of a set
  if (C::WM == 1 || set == 0)
    named_barrier(1, C::WN * 32);
  else
    named_barrier(2, C::WN * 32);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    chunk_rows_kernel(const __grid_constant__ PartialParams p, const __grid_constant__ ChunkMaps maps) {
  const CUtensorMap &tmk = maps.k, &tmv = maps.v;
  constexpr int D = C::D, TN = C::TN, NSTAGE = C::NSTAGE, WN = C::WN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NFULL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NFULL; ++s) mbar_init(&full[s], 1);
    for (int s = 0; s < NSTAGE; ++s) mbar_init(&empty[s], C::WM);
    fence_mbar_init();
  }
  // The second pass of a shared prefix starts under the end of the first (its merge), whose result it reads
  // at the end of an item only; the groups' arrays were complete before the first pass's attention
  // kernel began.  Every thread waits before it leaves, so that what comes after this grid may rely on the first
  // pass as well.
  auto first_pass_done = [&]() {
    if constexpr (C::SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (C::SHARED && p.ck.whole) first_pass_done();  // (the first pass itself: the groups' arrays)
  using Runs = ChunkRuns<C::SHARED>;
  Runs runs;  // (synchronises the block)
  if (!chunk_find_runs<C::THREADS, C::SHARED>(p.ck, gridDim.x, blockIdx.x, &runs)) {
    first_pass_done();
    return;
  }

  if (warp == C::WM * WN) {
    // ------------------------------------------------------------ producer warp
    // Pages and rows of 32 tiles at a time, a lane each: one tile's look-up after the other took as
    // long as a tile of codes
    if (lane == 0) {
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
    }
    const uint64_t pol = l2_policy_evict_first();
    int x = 0;  // tiles loaded
    ChunkPiece pc;
    bool ok = true;
    while (ok && runs.next(p.ck, &pc)) {
      for (int i0 = 0; ok && i0 < pc.n_tiles; i0 += 32) {
        int pages = 0, rows = 0;
        if (i0 + lane < pc.n_tiles) {
          const int t = pc.token(i0 + lane);
          pages = chunk_page_of<C::SHARED>(p, pc.b, t);
          rows = t % p.block_len;
        }
        const int n = min(32, pc.n_tiles - i0);
        for (int i = 0; i < n; ++i) {
          const int page = __shfl_sync(0xffffffffu, pages, i), row = __shfl_sync(0xffffffffu, rows, i);
          const int s = x % NSTAGE;
          if (lane == 0) {
            ok = x < NSTAGE || mbar_wait(&empty[s], ((x / NSTAGE) - 1) & 1, p.err, kDevErrEmptyWait);
            if (ok) {
              uint64_t* fb = &full[full_slot<C>(x)];
              mbar_arrive_expect_tx(fb, C::STAGE);
              uint8_t* ks = smem + s * C::STAGE;
#pragma unroll
              for (int bx = 0; bx < C::NBOX; ++bx) {
                tma_load_4d(ks + bx * C::BOX_BYTES, &tmk, fb, bx * C::BOX_ELEMS, row, pc.g, page, pol);
                tma_load_4d(ks + C::TILE + bx * C::BOX_BYTES, &tmv, fb, bx * C::BOX_ELEMS, row, pc.g, page, pol);
              }
              if constexpr (C::FP4) {
                tma_load_4d(ks + 2 * C::TILE, &maps.k_block, fb, row * (D / kFp4Block / 4), pc.g, page, 0, pol);
                tma_load_4d(ks + 2 * C::TILE + C::SCALES, &maps.v_block, fb, row * (D / kFp4Block / 4), pc.g, page, 0, pol);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          ++x;
        }
      }
    }
    // every issued copy lands before the CTA may exit
    for (int y = max(0, x - NSTAGE); y < x; ++y)
      if (!mbar_wait(&full[full_slot<C>(y)], full_parity<C>(y), p.err, kDevErrDrainWait)) break;
    first_pass_done();
    return;
  }

  // -------------------------------------------------------------- consumer warps
  const int wm = C::WM == 1 ? 0 : warp / WN, wn = warp - wm * WN;
  const int gq = lane >> 2, tq = lane & 3;
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML) + wm * WN * kRows * 2;
  uint4* qfrag = reinterpret_cast<uint4*>(smem + C::OFF_QF) + wm * (D / 16) * 32;
  float* q_scale = reinterpret_cast<float*>(smem + C::OFF_QS) + wm * kRows;
  // the run and its piece wait in shared memory: the registers are full of scores and O
  static_assert(sizeof(Runs) <= 64 && sizeof(ChunkPiece) <= 128, "a warp's place");
  Runs* run = reinterpret_cast<Runs*>(smem + C::OFF_RUN + warp * 192);
  ChunkPiece& pc = *reinterpret_cast<ChunkPiece*>(smem + C::OFF_RUN + warp * 192 + 64);
  if (lane == 0) *run = runs;
  auto next_piece = [&]() -> bool {
    __syncwarp();  // the piece's readers are done
    bool more = false;
    if (lane == 0) more = run->next(p.ck, &pc);
    more = __any_sync(0xffffffffu, more);
    __syncwarp();  // lane 0's stores
    return more;
  };
  int x0 = 0;  // tiles of the pieces before
  // A warp that gave up a wait takes no further tile, but goes on through the pieces, since the
  // others of its set count on it at their barriers
  WarpWait wait(p.err);
  while (next_piece()) {
    const int rows_total = pc.n * p.G;
    const int mset = pc.mt * C::ROWS + wm * kRows;  // this set's first row
    const int mrow0 = mset + gq, mrow1 = mrow0 + 8;
    const bool v0 = mrow0 < rows_total, v1 = mrow1 < rows_total;
    const int tq0 = v0 ? mrow0 / p.G : 0, tq1 = v1 ? mrow1 / p.G : 0;
    const int h0 = pc.g * p.G + (v0 ? mrow0 % p.G : 0), h1 = pc.g * p.G + (v1 ? mrow1 % p.G : 0);
    // visible tokens of a row: [wl, hz] and below the sinks' end; all below the item's end
    const int pos0 = chunk_pos0<C::SHARED>(p.ck, pc.n, pc.m), pos_step = chunk_pos_step<C::SHARED>(p.ck);
    const int hz0 = pos0 + tq0 * pos_step, hz1 = pos0 + tq1 * pos_step, hz_min = pos0 + mset / p.G * pos_step;
    auto window_lo = [&](int pos) -> int { return p.ck.window > 0 && pos >= p.ck.window ? pos - p.ck.window + 1 : 0; };
    const int wl0 = window_lo(hz0), wl1 = window_lo(hz1);
    const int wl_max = window_lo(pos0 + min(mset + kRows - 1, rows_total - 1) / p.G);
    const bool idle = C::WM > 1 && mset >= rows_total;  // a set without rows only passes the tiles on

    // ---- Q fragments (A operand, 16 rows x D): registers for bf16, shared memory for fp8
    uint32_t qa[C::CODES ? 1 : D / 16][4];
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + pc.row0 * p.q_st;
      const __nv_bfloat16* q0 = q + tq0 * p.q_st + h0 * p.q_sh;
      const __nv_bfloat16* q1 = q + tq1 * p.q_st + h1 * p.q_sh;
      if constexpr (!C::CODES) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int d0 = 16 * ks + 2 * tq;
          qa[ks][0] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + d0) : 0u;
          qa[ks][1] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + d0) : 0u;
          qa[ks][2] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + d0 + 8) : 0u;
          qa[ks][3] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + d0 + 8) : 0u;
        }
      } else {
        // A row times the power of two that puts its largest magnitude in [2^14, 2^15) converts to fp16
        // without overflow, exactly for every element within 2^-31 of the largest; the power goes back
        // into the row's score scale (NaN for a row with an infinity or a NaN, which says the same of the
        // row and nothing of the others)
        consumers_sync<C>(wm);  // the fragments' readers of the piece before are done
        if (wn == 0) {
          uint2 u[2][D / 16];
          uint32_t most[2] = {0u, 0u};  // magnitudes order as their bits
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            // k-slots (2tq, 2tq+1 | 2tq+8, 2tq+9) hold d = 16ks + 4tq + (0,1 | 2,3), the order in
            // which ldmatrix delivers the e4m3 key bytes
            // (4-bit: of a chunk of 32 dims the lane has 8 tq .. 8 tq + 7, half for each step)
            const int d0 = C::FP4 ? 32 * (ks >> 1) + 8 * tq + 4 * (ks & 1) : 16 * ks + 4 * tq;
            u[0][ks] = v0 ? *reinterpret_cast<const uint2*>(q0 + d0) : make_uint2(0u, 0u);
            u[1][ks] = v1 ? *reinterpret_cast<const uint2*>(q1 + d0) : make_uint2(0u, 0u);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (uint32_t w : {u[r][ks].x, u[r][ks].y})
                most[r] = max(most[r], max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
          }
          float down[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {  // a row's lanes: 4 gq .. 4 gq + 3
            most[r] = max(most[r], __shfl_xor_sync(0xffffffffu, most[r], 1));
            most[r] = max(most[r], __shfl_xor_sync(0xffffffffu, most[r], 2));
            const bool finite = most[r] < 0x7F800000u;
            const int qe = most[r] == 0u ? 0 : min(max(static_cast<int>(most[r] >> 23) - 127 - 14, -126), 126);
            down[r] = __uint_as_float(static_cast<uint32_t>(127 - qe) << 23);
            if (tq == 0)
              q_scale[gq + 8 * r] =
                  finite ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + qe) << 23) : __int_as_float(0x7fc00000);
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            qfrag[ks * 32 + lane] = make_uint4(pack_f16(bf16_lo(u[0][ks].x) * down[0], bf16_hi(u[0][ks].x) * down[0]),
                                               pack_f16(bf16_lo(u[1][ks].x) * down[1], bf16_hi(u[1][ks].x) * down[1]),
                                               pack_f16(bf16_lo(u[0][ks].y) * down[0], bf16_hi(u[0][ks].y) * down[0]),
                                               pack_f16(bf16_lo(u[1][ks].y) * down[1], bf16_hi(u[1][ks].y) * down[1]));
        }
        consumers_sync<C>(wm);
      }
    }

    const float k_head = C::FP4 ? head_scale(p.k_head, pc.g) : 1.f;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mrun[2] = {-INFINITY, -INFINITY};
    float lrun[2] = {0.f, 0.f};
    // fp8: p times the V scale goes to fp16, whose 11 bits hold from 2^-14 to 2^16, so each row has a
    // power of two, up, by which its weights and its O are multiplied: the largest weight of a tile lies
    // between 2^4 and 2^15 then, and what is above 2^-28 of it (2^-18 where it lies lowest) keeps its
    // bits, however far apart the scales and the scores of the row's tiles are
    // (4-bit pages: the scales are in V's own values, so the weights need no more than a power that puts
    // the largest possible one, that of the running maximum, at 2^kUp4: a weight keeps all bits down to 2^-28 of
    // it and counts down to 2^-38, so that even 2^20 tokens below that miss 2^-18)
    constexpr float kUp4 = 14.f;
    constexpr int kMostUp = 124;  // (2^-kMostUp is a normal number)
    float up[2];
    up[0] = up[1] = __uint_as_float(static_cast<uint32_t>(127 + kMostUp) << 23);

    // this warp's tiles: those whose number in the CTA is wn modulo WN
    for (int i = (wn + WN - x0 % WN) % WN; i < pc.n_tiles; i += WN) {
      const int x = x0 + i, s = x % NSTAGE;
      const int t0 = pc.token(i);
      float ksc = 1.f, vsc = 1.f;
      if constexpr (C::FP8) {
        // a page outside the cache reads as zeros through TMA; its scale is never fetched
        const int page = chunk_page_of<C::SHARED>(p, pc.b, t0);
        ksc = vsc = 0.f;
        if (page >= 0 && page < p.num_blocks) {
          const int per = p.block_len / p.scale_block;
          const int64_t idx = (static_cast<int64_t>(page) * p.Hkv + pc.g) * per + (t0 % p.block_len) / p.scale_block;
          ksc = __ldg(p.k_scale + idx);
          vsc = __ldg(p.v_scale + idx);
        }
      }
      if (!wait(&full[full_slot<C>(x)], full_parity<C>(x), kDevErrFullWait)) break;
      if (idle) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        continue;
      }
      const uint32_t kbase = smem_u32(smem + s * C::STAGE);
      const uint32_t vbase = kbase + C::TILE;
      const int mi = lane >> 3;

      // ---- S = Q K^T  (16 x 64)
      float sc[TN / 8][4];
#pragma unroll
      for (int i2 = 0; i2 < TN / 8; ++i2) sc[i2][0] = sc[i2][1] = sc[i2][2] = sc[i2][3] = 0.f;
      if constexpr (!C::CODES) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
          for (int np = 0; np < TN / 16; ++np) {
            const uint32_t tok = 16 * np + (mi >> 1) * 8 + (lane & 7);
            const uint32_t byte = (2 * ks + (mi & 1)) * 16;
            uint32_t r0, r1, r2, r3;
            ldsm_x4(kbase + tile_off<C>(tok, byte), r0, r1, r2, r3);
            mma_bf16(sc[2 * np], qa[ks], r0, r1);
            mma_bf16(sc[2 * np + 1], qa[ks], r2, r3);
          }
        }
      } else if constexpr (C::FP4) {
        // Of 8 tokens a lane has token gq, of each chunk of 32 dims 8 tq .. 8 tq + 7, which lie in one
        // block.  Code times block scale is exact in fp16 (6 bits, 2^-10 to 2688).  Two chunks at a
        // time: their queries stay in registers over the tile's tokens
        const uint8_t* ksb = smem + s * C::STAGE + 2 * C::TILE + gq * (D / kFp4Block);
#pragma unroll
        for (int c2 = 0; c2 < D / 64; ++c2) {
          uint4 qv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) qv[i] = qfrag[(4 * c2 + i) * 32 + lane];
#pragma unroll
          for (int np = 0; np < TN / 16; np += 2) {
            uint32_t w[4][2];  // [8 tokens][chunk]
#pragma unroll
            for (int h = 0; h < 4; h += 2)
              ldsm_x4(kbase + tile4_off(16 * np + (h + (mi >> 1)) * 8 + (lane & 7), (2 * c2 + (mi & 1)) * 16), w[h][0], w[h][1],
                      w[h + 1][0], w[h + 1][1]);
            uint32_t by[4];  // the scales of the two chunks' blocks
#pragma unroll
            for (int h = 0; h < 4; ++h)
              by[h] = e4m3x2_low_to_f16x2(prmt(
                  ring_load(ksb + (16 * np + 8 * h) * (D / kFp4Block) + 4 * c2), 0u, (tq >> 1) ? 0x31u : 0x20u));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t qa0[4] = {qv[2 * c].x, qv[2 * c].y, qv[2 * c].z, qv[2 * c].w};
              const uint32_t qa1[4] = {qv[2 * c + 1].x, qv[2 * c + 1].y, qv[2 * c + 1].z, qv[2 * c + 1].w};
              uint32_t k[4][4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const uint32_t b = prmt(by[h], 0u, c ? 0x3232u : 0x1010u);
                e2m1x8_to_f16x2x4(w[h][c], k[h][0], k[h][1], k[h][2], k[h][3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) k[h][j] = mul_f16x2(k[h][j], b);
              }
              // (four independent products between two into the same scores)
#pragma unroll
              for (int h = 0; h < 4; ++h) mma_f16(sc[2 * np + h], qa0, k[h][0], k[h][1]);
#pragma unroll
              for (int h = 0; h < 4; ++h) mma_f16(sc[2 * np + h], qa1, k[h][2], k[h][3]);
            }
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2) {
          const uint4 qv0 = qfrag[ks * 32 + lane];
          const uint4 qv1 = qfrag[(ks + 1) * 32 + lane];
          const uint32_t qa0[4] = {qv0.x, qv0.y, qv0.z, qv0.w};
          const uint32_t qa1[4] = {qv1.x, qv1.y, qv1.z, qv1.w};
#pragma unroll
          for (int np = 0; np < TN / 16; ++np) {
            const uint32_t tok = 16 * np + (mi >> 1) * 8 + (lane & 7);
            const uint32_t byte = (ks + (mi & 1)) * 16;
            uint32_t r0, r1, r2, r3;
            ldsm_x4(kbase + tile_off<C>(tok, byte), r0, r1, r2, r3);
            uint32_t k0l, k0h, k1l, k1h, k2l, k2h, k3l, k3h;
            e4m3x4_to_f16x2x2(r0, k0l, k0h);
            e4m3x4_to_f16x2x2(r1, k1l, k1h);
            e4m3x4_to_f16x2x2(r2, k2l, k2h);
            e4m3x4_to_f16x2x2(r3, k3l, k3h);
            mma_f16(sc[2 * np], qa0, k0l, k0h);
            mma_f16(sc[2 * np], qa1, k1l, k1h);
            mma_f16(sc[2 * np + 1], qa0, k2l, k2h);
            mma_f16(sc[2 * np + 1], qa1, k3l, k3h);
          }
        }
      }

      // ---- scale, mask, online softmax
      float sl[2] = {p.scale_log2, p.scale_log2};
      if constexpr (C::CODES) {
        if constexpr (C::FP4) ksc = k_head;
        sl[0] = reinterpret_cast<volatile const float*>(q_scale)[gq] * ksc;
        sl[1] = reinterpret_cast<volatile const float*>(q_scale)[gq + 8] * ksc;
      }
      // tokens of this tile that some row of the item sees / that every row of it sees
      const int r_lo = pc.tl.lo, r_hi = pc.tl.hi, sinks = pc.tl.sinks;
      const bool in_range = (t0 >= r_lo && t0 + TN <= r_hi) || t0 + TN <= sinks;
      const bool need_mask = !in_range || t0 + TN - 1 > hz_min || (t0 < wl_max && t0 + TN > sinks);
      auto in_item = [&](int tok) -> bool { return (tok >= r_lo && tok < r_hi) || tok < sinks; };
      float tmax[2] = {-INFINITY, -INFINITY};
      // an instantiation per mask mode: most tiles carry no test
      // (4-bit: packed arithmetic, here and below)
      auto scale_all = [&]() {
#pragma unroll
        for (int nt = 0; nt < TN / 8; ++nt) {
          mul_pair(sc[nt][0], sc[nt][1], sl[0]);
          mul_pair(sc[nt][2], sc[nt][3], sl[1]);
          tmax[0] = fmax3(tmax[0], sc[nt][0], sc[nt][1]);
          tmax[1] = fmax3(tmax[1], sc[nt][2], sc[nt][3]);
        }
      };
      auto scale_mask = [&](auto masked) {
#pragma unroll
        for (int nt = 0; nt < TN / 8; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = sc[nt][e] * sl[e >> 1];
            if constexpr (decltype(masked)::value) {
              const int tok = t0 + 8 * nt + 2 * tq + (e & 1);
              const bool seen = tok < r_hi && tok <= ((e < 2) ? hz0 : hz1) &&
                                (tok >= ((e < 2) ? wl0 : wl1) || tok < sinks);
              y = seen ? y : -INFINITY;
            }
            sc[nt][e] = y;
            tmax[e >> 1] = fmaxf(tmax[e >> 1], y);
          }
        }
      };
      if (need_mask)
        scale_mask(std::true_type{});
      else if constexpr (C::FP4)
        scale_all();
      else
        scale_mask(std::false_type{});
      // (base: what scores are taken against)
      float base[2], alpha[2], fall[2], vs[2] = {1.f, 1.f};
      bool other = false;  // fp8: a row's largest weight leaves its range
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], 1));
        tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], 2));
        const float mnew = fmaxf(mrun[r], tmax[r]);
        base[r] = (mnew == -INFINITY) ? 0.f : mnew;
        fall[r] = mrun[r] - base[r];
        alpha[r] = fast_exp2(fall[r]);  // 0 when mrun = -inf
        mrun[r] = mnew;
        lrun[r] *= alpha[r];
        if constexpr (C::FP8) {
          vs[r] = vsc * up[r];
          const float most = fabsf(vs[r]) * fast_exp2(tmax[r] - base[r]);
          other = other || !(most >= 16.f && most <= 32768.f);
        }
      }
      if constexpr (C::FP8) {
        if (__any_sync(0xffffffffu, other)) {
          // log2 of a row's largest weight in this tile (below 2^-100 of its scale it is nothing), and of up
          const int e = static_cast<int>((__float_as_uint(vsc) >> 23) & 0xFFu) - 127;
          float most[2];
          int was[2], to[2];
          bool lower = false;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            most[r] = static_cast<float>(e) + fmaxf(tmax[r] - base[r], -100.f);
            was[r] = static_cast<int>(__float_as_uint(up[r]) >> 23) - 127;
            to[r] = min(14 - static_cast<int>(ceilf(most[r])), kMostUp);
            // (a row that sees nothing here keeps its power; its weights are zeros, whatever the scale)
            if (tmax[r] == -INFINITY || vsc == 0.f || (to[r] >= was[r] && to[r] <= was[r] + 8)) to[r] = was[r];
            lower = lower || to[r] > was[r];
          }
          if (__any_sync(0xffffffffu, lower)) {
            // O grows with its power, up to 2^100: the largest of each row's O (a thread's columns are rows
            // 2tq, 2tq+1 (+8); the other lanes of the same rows hold other dims)
            float big[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int i2 = 0; i2 < D / 8; ++i2)
#pragma unroll
              for (int q = 0; q < 4; ++q) big[i2 & 1][q & 1] = fmaxf(big[i2 & 1][q & 1], fabsf(o[i2][q]));
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) big[r][q] = fmaxf(big[r][q], __shfl_xor_sync(0xffffffffu, big[r][q], w));
              const float even = __shfl_sync(0xffffffffu, big[r][0], gq >> 1), odd = __shfl_sync(0xffffffffu, big[r][1], gq >> 1);
              const float x = (gq & 1) ? odd : even;
              const float room = 100.f - (static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 126) + fall[r]);
              if (to[r] > was[r] && x > 0.f) to[r] = min(to[r], was[r] + max(static_cast<int>(fminf(room, 300.f)), 0));
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (to[r] != was[r]) alpha[r] = fast_exp2(fall[r] + static_cast<float>(to[r] - was[r]));
            up[r] = __uint_as_float(static_cast<uint32_t>(127 + to[r]) << 23);
            vs[r] = tmax[r] == -INFINITY ? 0.f : vsc * up[r];
          }
        }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {  // a row max (or its power) moved
        if constexpr (!C::CODES) {
#pragma unroll
          for (int i2 = 0; i2 < D / 8; ++i2) {
            o[i2][0] *= alpha[0];
            o[i2][1] *= alpha[0];
            o[i2][2] *= alpha[1];
            o[i2][3] *= alpha[1];
          }
        } else {
          // O^T: this thread's columns are rows 2tq, 2tq+1 (+8)
          float ar[2][2];
          ar[0][0] = __shfl_sync(0xffffffffu, alpha[0], 8 * tq);
          ar[0][1] = __shfl_sync(0xffffffffu, alpha[0], 8 * tq + 4);
          ar[1][0] = __shfl_sync(0xffffffffu, alpha[1], 8 * tq);
          ar[1][1] = __shfl_sync(0xffffffffu, alpha[1], 8 * tq + 4);
#pragma unroll
          for (int i2 = 0; i2 < D / 8; ++i2) {
            const int n = i2 & 1;
            o[i2][0] *= ar[n][0];
            o[i2][1] *= ar[n][1];
            o[i2][2] *= ar[n][0];
            o[i2][3] *= ar[n][1];
          }
        }
      }
      uint32_t pa[TN / 16][4];
      if constexpr (C::FP4) {
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int nt = 0; nt < TN / 8; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // (two steps: a very large maximum less kUp4 would be rounded, and not alike in all warps)
            add_pair(sc[nt][2 * r], sc[nt][2 * r + 1], -base[r]);
            add_pair(sc[nt][2 * r], sc[nt][2 * r + 1], kUp4);
            const float p0 = fast_exp2(sc[nt][2 * r]), p1 = fast_exp2(sc[nt][2 * r + 1]);
            sum[r] = add_f32x2(sum[r], p0, p1);
            pa[nt >> 1][(nt & 1) * 2 + r] = pack_f16(p0, p1);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) lrun[r] += sum_f32x2(sum[r]);
      }
#pragma unroll
      for (int nt = 0; nt < (C::FP4 ? 0 : TN / 8); ++nt) {
        const float p0 = fast_exp2(sc[nt][0] - base[0]);
        const float p1 = fast_exp2(sc[nt][1] - base[0]);
        const float p2 = fast_exp2(sc[nt][2] - base[1]);
        const float p3 = fast_exp2(sc[nt][3] - base[1]);
        lrun[0] += p0 + p1;
        lrun[1] += p2 + p3;
        const int kk = nt >> 1, hf = (nt & 1) * 2;
        if constexpr (!C::CODES) {
          pa[kk][hf + 0] = pack_bf16(p0, p1);
          pa[kk][hf + 1] = pack_bf16(p2, p3);
        } else {
          pa[kk][hf + 0] = pack_f16(p0 * vs[0], p1 * vs[0]);
          pa[kk][hf + 1] = pack_f16(p2 * vs[1], p3 * vs[1]);
        }
      }

      // ---- O += P V; V rows that no row sees may hold anything: masked in the tiles that have some
      auto pv = [&](auto vmasked) {
#pragma unroll
        for (int kk = 0; kk < TN / 16; ++kk) {
          uint32_t mlo = 0xFFFFFFFFu, mhi = 0xFFFFFFFFu;
          if constexpr (decltype(vmasked)::value) {
            const int ta = t0 + 16 * kk + 2 * tq, tb = ta + 8;
            mlo = half_mask(in_item(ta), in_item(ta + 1));
            mhi = half_mask(in_item(tb), in_item(tb + 1));
          }
          if constexpr (!C::CODES) {
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
              const uint32_t tok = 16 * kk + (mi & 1) * 8 + (lane & 7);
              const uint32_t byte = (2 * dp + (mi >> 1)) * 16;
              uint32_t r0, r1, r2, r3;
              ldsm_x4_t(vbase + tile_off<C>(tok, byte), r0, r1, r2, r3);
              if constexpr (decltype(vmasked)::value) r0 &= mlo, r1 &= mhi, r2 &= mlo, r3 &= mhi;
              mma_bf16(o[2 * dp], pa[kk], r0, r1);
              mma_bf16(o[2 * dp + 1], pa[kk], r2, r3);
            }
          } else if constexpr (C::FP4) {
            // as below, 4 dims of two tokens a lane: of dims 32 c + 4 gq + i the nibbles of both tokens
            // make one byte, and so one pair.  Row gq of the product's tiles 2 c and 2 c + 1 is
            // dim 4 gq or 4 gq + 2, row gq + 8 the next one
            const uint32_t b00 = pa[kk][0], b01 = pa[kk][2], b10 = pa[kk][1], b11 = pa[kk][3];
            const uint8_t* vsb = smem + s * C::STAGE + 2 * C::TILE + C::SCALES + (16 * kk + 2 * tq) * (D / kFp4Block);
            const uint4 sa = ring_load_v4(vsb);  // two tokens' scales
            const uint4 sb = ring_load_v4(vsb + 8 * (D / kFp4Block));
            uint32_t sv[2][4];  // scales of the pairs of tokens, blocks 2 c + (gq >> 2)
            {
              const uint32_t sel = (gq >> 2) ? 0x7351u : 0x6240u;  // (t0, t1) of a word's first, then second block
              e4m3x4_to_f16x2x2(prmt(sa.x, sa.z, sel), sv[0][0], sv[0][1]);
              e4m3x4_to_f16x2x2(prmt(sa.y, sa.w, sel), sv[0][2], sv[0][3]);
              e4m3x4_to_f16x2x2(prmt(sb.x, sb.z, sel), sv[1][0], sv[1][1]);
              e4m3x4_to_f16x2x2(prmt(sb.y, sb.w, sel), sv[1][2], sv[1][3]);
            }
            auto pairs = [](uint32_t w, uint32_t* f) {  // dims 0, 1, 2, 3 of both tokens
              // one token's nibble under the other's: dims 0 and 2 in the low half, 1 and 3 in the high one
              const uint32_t moved = prmt(w >> 12, w << 12, 0x7610u);
              e2m1x8_to_f16x2x4((w & 0xF0F00F0Fu) | (moved & 0x0F0FF0F0u), f[0], f[2], f[1], f[3]);
            };
            uint32_t w[2][2];  // [chunk & 1][8 tokens]
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              if ((c & 1) == 0)
                ldsm_x4_t(vbase + tile4_off(16 * kk + (mi & 1) * 8 + (lane & 7), (c + (mi >> 1)) * 16), w[0][0], w[0][1], w[1][0],
                          w[1][1]);
              uint32_t f[2][4];
              pairs(w[c & 1][0], f[0]);
              pairs(w[c & 1][1], f[1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f[0][i] = mul_f16x2(f[0][i], sv[0][c]);
                f[1][i] = mul_f16x2(f[1][i], sv[1][c]);
                if constexpr (decltype(vmasked)::value) f[0][i] &= mlo, f[1][i] &= mhi;  // (the scales may be anything too)
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a[4] = {f[0][2 * i], f[0][2 * i + 1], f[1][2 * i], f[1][2 * i + 1]};
                mma_f16(o[2 * (2 * c + i)], a, b00, b01);
                mma_f16(o[2 * (2 * c + i) + 1], a, b10, b11);
              }
            }
          } else {
            // O^T[dv x rows] += V^T[dv x tok] P^T[tok x rows]: ldmatrix.trans of the e4m3 tile
            // (16-bit view) gives each lane two tokens x two dims, one byte permute pairs them by
            // dim, and P's fragments are the B operand as they are
            const uint32_t b00 = pa[kk][0], b01 = pa[kk][2], b10 = pa[kk][1], b11 = pa[kk][3];
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) {
              const uint32_t tok = 16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7);
              uint32_t r0, r1;
              ldsm_x2_t(vbase + tile_off<C>(tok, cc * 16), r0, r1);
              uint32_t a[4];
              if constexpr (decltype(vmasked)::value) r0 &= mlo, r1 &= mhi;
              e4m3x4_to_f16x2x2(prmt(r0, 0u, 0x3120u), a[0], a[1]);
              e4m3x4_to_f16x2x2(prmt(r1, 0u, 0x3120u), a[2], a[3]);
              mma_f16(o[2 * cc], a, b00, b01);
              mma_f16(o[2 * cc + 1], a, b10, b11);
            }
          }
        }
      };
      if (in_range)
        pv(std::false_type{});
      else
        pv(std::true_type{});
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    x0 += pc.n_tiles;

    // ---- join the warps: (m, l) of every row first, then O warp by warp into the first one
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      lrun[r] += __shfl_xor_sync(0xffffffffu, lrun[r], 1);
      lrun[r] += __shfl_xor_sync(0xffffffffu, lrun[r], 2);
      if (tq == 0) {
        ml[(wn * kRows + gq + 8 * r) * 2] = mrun[r];
        ml[(wn * kRows + gq + 8 * r) * 2 + 1] = lrun[r];
      }
    }
    consumers_sync<C>(wm);
    float M[2], L[2], f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      M[r] = -INFINITY;
#pragma unroll
      for (int w = 0; w < WN; ++w) M[r] = fmaxf(M[r], ml[(w * kRows + gq + 8 * r) * 2]);
      const float base = M[r] == -INFINITY ? 0.f : M[r];
      L[r] = 0.f;  // a NaN among the scores keeps it NaN, and the row is NaN
#pragma unroll
      for (int w = 0; w < WN; ++w) L[r] += ml[(w * kRows + gq + 8 * r) * 2 + 1] * fast_exp2(ml[(w * kRows + gq + 8 * r) * 2] - base);
      f[r] = fast_exp2(mrun[r] - base);
      if constexpr (C::FP8) f[r] *= __uint_as_float((254u << 23) - __float_as_uint(up[r]));  // 1 / up
      if constexpr (C::FP4) f[r] *= head_scale(p.v_head, pc.g);
      // (a warp without a tile has O = 0; 0 * 2^-inf = 0)
    }
    // the factor of each element: rows gq, gq + 8; fp8: O^T, rows 2tq, 2tq+1 (+8)
    float fr[4] = {f[0], f[0], f[1], f[1]};
    if constexpr (C::CODES) {
      fr[0] = __shfl_sync(0xffffffffu, f[0], 8 * tq);
      fr[1] = __shfl_sync(0xffffffffu, f[0], 8 * tq + 4);
      fr[2] = __shfl_sync(0xffffffffu, f[1], 8 * tq);
      fr[3] = __shfl_sync(0xffffffffu, f[1], 8 * tq + 4);
    }
#pragma unroll
    for (int i2 = 0; i2 < D / 8; ++i2)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i2][e] *= C::CODES ? fr[2 * (i2 & 1) + (e & 1)] : fr[e];
    float4* obuf = reinterpret_cast<float4*>(smem + C::OFF_O) + wm * (D / 8) * 32;
#pragma unroll 1
    for (int w = 1; w < WN; ++w) {
      if (wn == w) {
#pragma unroll
        for (int i2 = 0; i2 < D / 8; ++i2) obuf[i2 * 32 + lane] = make_float4(o[i2][0], o[i2][1], o[i2][2], o[i2][3]);
      }
      consumers_sync<C>(wm);
      if (wn == 0) {
#pragma unroll
        for (int i2 = 0; i2 < D / 8; ++i2) {
          const float4 y = obuf[i2 * 32 + lane];
          o[i2][0] += y.x, o[i2][1] += y.y, o[i2][2] += y.z, o[i2][3] += y.w;
        }
      }
      consumers_sync<C>(wm);
    }

    // ---- the first warp stores: final rows in bf16, or a partial (an empty one's o is never read)
    if (wn == 0) {
      constexpr float kLn2 = 0.6931471805599453f;
      const bool direct = pc.slot < 0;
      const int64_t row_a = direct ? (pc.row0 + static_cast<int64_t>(tq0)) * p.Hq + h0
                                   : static_cast<int64_t>(pc.slot) * C::ROWS + wm * kRows + gq;
      const int64_t row_b = direct ? (pc.row0 + static_cast<int64_t>(tq1)) * p.Hq + h1 : row_a + 8;
      const bool some0 = L[0] != 0.f, some1 = L[1] != 0.f;
      float inv0 = some0 ? 1.f / L[0] : 0.f, inv1 = some1 ? 1.f / L[1] : 0.f;
      const bool w0 = v0 && (some0 || direct), w1 = v1 && (some1 || direct);
      constexpr float kUp = C::FP4 ? kUp4 : 0.f;
      float lse0 = some0 ? (M[0] + (__log2f(L[0]) - kUp)) * kLn2 : -INFINITY;
      float lse1 = some1 ? (M[1] + (__log2f(L[1]) - kUp)) * kLn2 : -INFINITY;
      float prior0 = 0.f, prior1 = 0.f;  // weights of the prefix's result
      const bool behind = C::SHARED && direct && pc.skip > 0;
      if (behind) {
        first_pass_done();
        if (v0) {
          const ChunkJoin j = chunk_join(lse0, __ldcg(p.ck.prior_lse + row_a));
          inv0 *= j.own, prior0 = j.prior, lse0 = j.lse;
        }
        if (v1) {
          const ChunkJoin j = chunk_join(lse1, __ldcg(p.ck.prior_lse + row_b));
          inv1 *= j.own, prior1 = j.prior, lse1 = j.lse;
        }
      }
      const bool f32 = !direct || (C::SHARED && p.ck.out_f32);
      float* out_f = C::SHARED && direct ? static_cast<float*>(p.ck.out) : p.out_o;
      auto store2 = [&](int64_t row, int d, float y0, float y1) {
        if (f32)
          *reinterpret_cast<float2*>(out_f + row * D + d) = make_float2(y0, y1);
        else
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.ck.out) + row * D + d) = pack_bf16(y0, y1);
      };
      if constexpr (!C::CODES) {
        if constexpr (C::SHARED) {  // (loads in batches ahead of the stores: one after the other took 15 us an item)
#pragma unroll
          for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][e] *= e < 2 ? inv0 : inv1;
#pragma unroll
          for (int n0 = 0; n0 < D / 8; n0 += 8) {
            float2 x[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int d = 8 * (n0 + i) + 2 * tq;
              x[i] = y[i] = make_float2(0.f, 0.f);
              if (behind && v0) x[i] = __ldcg(reinterpret_cast<const float2*>(p.ck.prior_o + row_a * D + d));
              if (behind && v1) y[i] = __ldcg(reinterpret_cast<const float2*>(p.ck.prior_o + row_b * D + d));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* z = o[n0 + i];
              z[0] = fmaf(x[i].x, prior0, z[0]), z[1] = fmaf(x[i].y, prior0, z[1]);
              z[2] = fmaf(y[i].x, prior1, z[2]), z[3] = fmaf(y[i].y, prior1, z[3]);
            }
          }
          inv0 = inv1 = 1.f;
        }
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
          const int d = 8 * nt + 2 * tq;
          if (w0) store2(row_a, d, o[nt][0] * inv0, o[nt][1] * inv0);
          if (w1) store2(row_b, d, o[nt][2] * inv1, o[nt][3] * inv1);
        }
      } else {
        // O^T: this thread holds rows (8n + 2tq + {0,1}) at dv 16c + 2gq + {0,1}
        // (4-bit: 32 (c >> 1) + 4 gq + 2 (c & 1) + {0,1})
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int src = 4 * (2 * tq + e);
            const float inv = __shfl_sync(0xffffffffu, n ? inv1 : inv0, src);
            const bool wr = __shfl_sync(0xffffffffu, (n ? w1 : w0) ? 1 : 0, src) != 0;
            const int64_t row = __shfl_sync(0xffffffffu, n ? row_b : row_a, src);
            float2 x[D / 16];  // of the prefix, all loaded ahead of the stores
            if constexpr (C::SHARED) {
              const float prior = __shfl_sync(0xffffffffu, n ? prior1 : prior0, src);
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                const int d = C::FP4 ? 32 * (c >> 1) + 4 * gq + 2 * (c & 1) : 16 * c + 2 * gq;
                x[c] = make_float2(0.f, 0.f);
                if (behind && wr) x[c] = __ldcg(reinterpret_cast<const float2*>(p.ck.prior_o + row * D + d));
              }
#pragma unroll
              for (int c = 0; c < D / 16; ++c) x[c] = make_float2(x[c].x * prior, x[c].y * prior);
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const float* ov = o[2 * c + n];
              const int d = C::FP4 ? 32 * (c >> 1) + 4 * gq + 2 * (c & 1) : 16 * c + 2 * gq;
              if (!wr) continue;
              if constexpr (C::SHARED)
                store2(row, d, fmaf(ov[e], inv, x[c].x), fmaf(ov[2 + e], inv, x[c].y));
              else
                store2(row, d, ov[e] * inv, ov[2 + e] * inv);
            }
          }
        }
      }
      if (tq == 0) {
        float* lse = direct ? p.ck.lse : p.out_lse;
        if (v0) lse[row_a] = lse0;
        if (v1) lse[row_b] = lse1;
      }
    }
    // (the next piece writes ml and obuf behind a sync that the first warp reaches after this)
  }
  first_pass_done();
}

// (4-bit, 16 rows: 5 warps 276 us for the 8 long sequences above where 4 took 252, 3 285)
// (two sets with bf16 heads of 128: 5 warps a set have 168 registers each, too few: 95 us for 24
// sequences of 5 rows, 40 / 8 heads, where 3 warps of 233 take 90; the other two fit, fp8 104 -> 90)
template <int WM, bool SHARED>
using CfgBf16D64 = RowsCfg<kPagesBf16, 64, WM, WM == 1 ? 4 : 5, WM == 1 ? 6 : 12, SHARED>;
template <int WM, bool SHARED>
using CfgBf16D128 = RowsCfg<kPagesBf16, 128, WM, 3, WM == 1 ? 3 : 6, SHARED>;
template <int WM, bool SHARED>
using CfgFp8D128 = RowsCfg<kPagesFp8, 128, WM, WM == 1 ? 4 : 5, WM == 1 ? 6 : 12, SHARED>;
template <int WM, bool SHARED>
using CfgFp4D128 = RowsCfg<kPagesFp4, 128, WM, WM == 1 ? 4 : 5, WM == 1 ? 8 : 15, SHARED>;

template <class C>
cudaError_t launch_cfg(const PartialParams& p, const ChunkMaps& maps, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};  // per variant, per device
  cudaError_t e0 = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(chunk_rows_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e0 != cudaSuccess) return e0;
  if constexpr (C::SHARED) {  // a programmatic dependent of the kernel before, which it waits for
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned int>(p.ck.n_wave));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_rows_kernel<C>, p, maps);
  }
  chunk_rows_kernel<C><<<static_cast<unsigned int>(p.ck.n_wave), C::THREADS, C::SMEM, stream>>>(p, maps);
  return cudaGetLastError();
}

template <int WM, bool SHARED>
cudaError_t launch_sets(const PartialParams& p, int32_t d, PageFormat pages, const ChunkMaps& maps, cudaStream_t stream) {
  if (pages == kPagesFp4) return launch_cfg<CfgFp4D128<WM, SHARED>>(p, maps, stream);
  if (pages == kPagesFp8) return launch_cfg<CfgFp8D128<WM, SHARED>>(p, maps, stream);
  if (d == 64) return launch_cfg<CfgBf16D64<WM, SHARED>>(p, maps, stream);
  return launch_cfg<CfgBf16D128<WM, SHARED>>(p, maps, stream);
}

}  // namespace

// (the passes of a shared prefix are compiled in a unit of their own, side by side with the others)
#ifdef SKV_CHUNK_SHARED
cudaError_t launch_chunk_rows_shared(const PartialParams& p, int32_t d, PageFormat pages, const ChunkMaps& maps,
                                     cudaStream_t stream) {
  return p.ck.rows == kRows ? launch_sets<1, true>(p, d, pages, maps, stream) : launch_sets<2, true>(p, d, pages, maps, stream);
}
#else
int chunk_rows_ctas_per_sm(int rows) { return rows == kRows ? 2 : 1; }

cudaError_t launch_chunk_rows(const PartialParams& p, int32_t d, PageFormat pages, const ChunkMaps& maps,
                              cudaStream_t stream) {
  if (p.ck.shared) return launch_chunk_rows_shared(p, d, pages, maps, stream);
  return p.ck.rows == kRows ? launch_sets<1, false>(p, d, pages, maps, stream) : launch_sets<2, false>(p, d, pages, maps, stream);
}
#endif

}  // namespace skv
