// Tensor-core (tcgen05) attention of ragged chunks of new tokens over a paged cache
// (attn_chunk_paged): prompt chunks, proposed tokens and decode tokens of one packed batch,
// causal or with a sliding window and sinks; bf16 pages, or fp8-e4m3 pages with block scales.
//
// For every row (new token at position p, query head h of KV head g): s_u = scale q.k_u over
// the visible tokens u (u <= p and u > p - window or u < n_sink), out = softmax(s) V, lse =
// ln sum e^s.  One pass over the tokens with a running maximum; sums and O in fp32, P rounded
// to bf16 for the product with V (2^-8 of each weight at most, as much as the output's own
// rounding).  O is divided by the fp32 sum of the unrounded weights: summing the rounded ones as
// well cost two more additions a pair of scores on the path that bounds the kernel.
//
// Bound by the tensor pipe for chunks of 128 and more rows (two 128 x 128 x D products per tile
// of 128 tokens and 128 rows), by HBM for few rows.  Design (one persistent CTA an SM, 384
// threads; warp 3 hands the work items to the other warps through shared memory):
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
//   * fp8: four converter warps split Q into two e4m3 parts (see split_q), so that Q K^T runs on the
//     K codes as they land, two 8-bit products at twice the rate, and widen the V codes to bf16
//     (exact) for P V; the K block scale goes into the score's scale, the V block scale into p
//     before its rounding.  (Widening K as well made the converters the bound: 554 us for ragged
//     prompts over an fp8 cache that take 329 this way);
//   * optimistic softmax: p = 2^(s - m) against the maximum so far; only a row's first visible
//     tile takes a maximum (of 32 columns) beforehand, and a tile whose p sum passes 2^16 its true
//     one, with O rescaled, and its p again.
#include <climits>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "chunk_plan.cuh"
#include "skv_common.cuh"
#include "skv_internal.h"
#include "tc_common.cuh"
#include "warp_wait.cuh"

namespace skv {

namespace {

constexpr int kTN = 128;        // tokens per K/V tile
constexpr int kHalf = kTN / 2;  // tokens per TMA box: a page holds a multiple of 64
constexpr int kRowsTile = 128;  // rows per query tile (MMA M)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S_k (P_k over its first 64 columns) at kColS + 128 k
constexpr uint32_t kColO = 256;  // O_k at kColO + 128 k
constexpr float kTileSumLimit = 65536.0f;
// Past this maximum (base 2) a score minus the maximum is taken after the score was rounded like it: the
// fused form leaves up to half a unit of the maximum's last place, which an exponential past 2^30 cannot hold
constexpr float kLargeScore = 4194304.0f;

template <int D_, bool FP8_>
struct TcCfg {
  static constexpr int D = D_;
  static constexpr bool FP8 = FP8_;
  static constexpr int THREADS = (FP8 ? 16 : 12) * 32;
  static constexpr int READERS = FP8 ? 15 : 11;      // warps that read the work items
  static constexpr int NB = D / 64;                  // 128-byte boxes of a row of 16-bit values
  static constexpr int NST = D == 64 ? 4 : 2;        // ring depth, tiles
  static constexpr int BOX = kTN * 128;              // one box column of a tile: 128 rows x 128 bytes
  static constexpr int TILE = NB * BOX;              // a Q or V tile of 128 rows in bf16
  static constexpr int LOAD = FP8 ? BOX : TILE;      // a K or V tile as it lands
  static constexpr int LOAD_BOXES = FP8 ? 1 : NB;
  static constexpr int LOAD_BOX_ELEMS = FP8 ? 128 : 64;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NST * LOAD;
  static constexpr int OFF_V8 = OFF_V + NST * TILE;  // fp8: the V codes' ring
  static constexpr int OFF_BAR = OFF_V8 + (FP8 ? NST * LOAD : 0);
  static constexpr int OFF_ML = OFF_BAR + 768;       // solo: group 1's (m, l) per row
  static constexpr int OFF_ITEM = OFF_ML + kRowsTile * 8;
  static constexpr int OFF_QS = OFF_ITEM + 256;      // fp8: Q's row scales [item & 1][query tile][row]
  static constexpr int OFF_OUT = OFF_QS + (FP8 ? 4 * kRowsTile * 4 : 0);  // 64 bytes of each output row
  static constexpr int OFF_ROW = OFF_OUT + 2 * kRowsTile * 64;            // what each softmax thread's row sees
  static constexpr int SMEM = 1024 + OFF_ROW + 2 * kRowsTile * 16;
  static_assert(kHalf == kTileN, "the plan counts in halves");
  static_assert(!FP8 || D == 128, "e4m3 rows are one 128-byte box");
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

constexpr int kScaleSlots = 8;  // tiles whose fp8 scales are held (see the loader)

template <class C>
struct TcBars {
  uint64_t item_full[2], item_empty[2];
  uint64_t q_full, q_empty;
  uint64_t k_full[C::NST], k_empty[C::NST];
  uint64_t v_full[C::NST], v_empty[C::NST];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t ml_full, o1_free;  // solo: group 1's (m, l) are written; group 0 has read them and O1
  // fp8: V codes have landed / are converted; Q is split (item & 1); a tile's scales are written
  uint64_t v8_full[C::NST], v8_empty[C::NST], q8_full[2], sc_full[kScaleSlots];
  float4 scales[kScaleSlots];  // K and V scale of a tile's first half, then of its second
  uint32_t tmem_base;
};

// What every role needs of a work item (written by the scheduling warp).
struct TcItem {
  ChunkItem it;
  ChunkTiles tl;
  int m0;       // first row of the row tile
  int pair;     // more than 128 rows
  int h0;       // first half of the chunk in tl's run
  int n_tiles;  // tiles of the chunk, two halves each
  // First token of the chunk's half h: tile i is the halves 2 i and 2 i + 1, which need not follow
  // one another (sinks and window; the last one may lie behind the run: no row sees its tokens).
  __device__ __forceinline__ int token(int h) const {
    const int x = h0 + h;
    return (x < tl.n_first ? x : tl.win + (x - tl.n_first)) * kHalf;
  }
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

// Four e4m3 codes to bf16, exactly.  A code's exponent and mantissa bits moved to a bf16's are
// the value times 2^(7 - 127) (a subnormal code becomes the subnormal bf16 of that product), so
// one packed multiplication by 2^120 gives the value: five operations a pair, where conversions
// by way of fp16 and fp32 take four of the slower conversion pipe's.  NaN codes come out as
// +-480 and are told by bit 7 of a byte of `odd`.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi, uint32_t& odd) {
  odd |= (w & 0x7F7F7F7Fu) + 0x01010101u;
  const __nv_bfloat162 k = __halves2bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80));  // 2^120
  const uint32_t a = prmt(w, 0u, 0x1404u), b = prmt(w, 0u, 0x3424u);  // codes in the high bytes
  uint32_t x = ((a >> 4) & 0x07F007F0u) | (a & 0x80008000u);
  uint32_t y = ((b >> 4) & 0x07F007F0u) | (b & 0x80008000u);
  __nv_bfloat162 u = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), k);
  __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&y), k);
  lo = *reinterpret_cast<uint32_t*>(&u);
  hi = *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
  return u;
}

// (x0, x1) * s for a pair in one packed instruction.
__device__ __forceinline__ void mul_pair(float& x0, float& x1, float s) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(s));
}

// An edge tile: the scores that this thread's row does not see (row: its end, the start of its
// window, the end of its sinks) become out0 (first half) or out1 in tensor memory, so that
// the passes over the scores carry no test.  hi_min, lo_max, sink_min: columns that the whole warp
// sees are left alone.  (A function of its own, as store_rows is: inlined, their registers spilled
// into the loop over the tiles, which then took 1.6 us a tile instead of 1.4.)
__device__ __noinline__ void hide_scores(uint32_t s_col, int ta, int tb, int4 row, int hi_min, int lo_max, int sink_min,
                                         float out0, float out1) {
#pragma unroll 1
  for (int c = 0; c < kTN; c += 32) {
    const int a = c < kHalf ? ta + c : tb + c - kHalf, b = a + 32;
    if (hi_min >= b && (lo_max <= a || sink_min >= b)) continue;  // all see all
    uint32_t x[2][16];
    tc::tmem_ld16(s_col + c, x[0]);
    tc::tmem_ld16(s_col + c + 16, x[1]);
    const uint32_t out = __float_as_uint(c < kHalf ? out0 : out1);
    uint32_t seen[2];  // bit e: column 16 h + e is seen
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = a + 16 * h;
      const int hi = min(max(row.x - f, 0), 16), lo = min(max(row.y - f, 0), 16), sink = min(max(row.z - f, 0), 16);
      seen[h] = ((1u << hi) - 1u) & ((0xFFFFu << lo) | ((1u << sink) - 1u));
    }
    tc::tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[h][e] = ((seen[h] >> e) & 1u) ? x[h][e] : out;
    tc::tmem_st16(s_col + c, x[0]);
    tc::tmem_st16(s_col + c + 16, x[1]);
  }
  tc::tmem_wait_st();
}

// The largest score (scaled) of 32 columns in tensor memory.
template <bool FP8>
__device__ __forceinline__ float largest(uint32_t s_col, float scale) {
  uint32_t x[2][16];
  tc::tmem_ld16(s_col, x[0]);
  tc::tmem_ld16(s_col + 16, x[1]);
  tc::tmem_wait_ld();
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float u = __uint_as_float(x[e >> 3][(2 * e) & 15]), v = __uint_as_float(x[e >> 3][(2 * e + 1) & 15]);
    if constexpr (FP8) u *= scale, v *= scale;  // (a block scale may be negative)
    m4[e & 3] = fmax3(m4[e & 3], u, v);
  }
  const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  return FP8 ? m : m * scale;
}

// A row's first visible tile (m = -inf) starts from the maximum of the first 32 columns that it
// sees: the limit on the p sum allows that to be 2^16 short.  Rows that do not exist go along where
// no mask tells them apart.
template <bool FP8>
__device__ __noinline__ float first_max(uint32_t s_col, float m, float scale0, float scale1) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int cc = 0; cc < kTN / 32; ++cc) {
    mx = fmaxf(mx, largest<FP8>(s_col + 32 * cc, cc < 2 ? scale0 : scale1));
    if (!__any_sync(0xffffffffu, m == -INFINITY && mx == -INFINITY)) break;
  }
  return m == -INFINITY ? mx : m;
}

// A tile in which the p sum of some row of the warp (need) passed the limit, or whose scores are very
// large: O and l rescaled to the tile's true maximum, and its P again.  PV of the group's tile before ran before these scores,
// so O is final.  l comes back with the tile's sum.
struct Redone {
  float m, l;
};
template <int D, bool FP8>
__device__ __noinline__ Redone redo_tile(uint32_t s_col, uint32_t o_col, bool need, float m, float l, float scale0,
                                         float scale1, float v0, float v1) {
  float mx = m;
#pragma unroll 1
  for (int cc = 0; cc < kTN / 32; ++cc) mx = fmaxf(mx, largest<FP8>(s_col + 32 * cc, cc < 2 ? scale0 : scale1));
  const float m_new = need ? mx : m;
  const float alpha = (need && l != 0.f) ? fast_exp2(m - m_new) : 1.f;
  if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t x[16];
      tc::tmem_ld16(o_col + c, x);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
      tc::tmem_st16(o_col + c, x);
    }
    tc::tmem_wait_st();
    l *= alpha;
  }
  const float base = (m_new == -INFINITY) ? 0.f : m_new;
  const bool large = fabsf(base) > kLargeScore;
  uint64_t ls[2] = {0ull, 0ull};
#pragma unroll 1
  for (int cc = 0; cc < kTN / 32; ++cc) {
    uint32_t x[2][16], w[16];
    tc::tmem_ld16(s_col + 32 * cc, x[0]);
    tc::tmem_ld16(s_col + 32 * cc + 16, x[1]);
    tc::tmem_wait_ld();
    const float s2 = cc < 2 ? scale0 : scale1, v2 = cc < 2 ? v0 : v1;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a0, a1;
      const float x0 = __uint_as_float(x[e >> 3][(2 * e) & 15]), x1 = __uint_as_float(x[e >> 3][(2 * e + 1) & 15]);
      fma_pair(x0, x1, s2, -base, a0, a1);
      if (large) a0 = __fadd_rn(__fmul_rn(x0, s2), -base), a1 = __fadd_rn(__fmul_rn(x1, s2), -base);
      float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
      ls[e & 1] = add_f32x2(ls[e & 1], p0, p1);
      if constexpr (FP8) mul_pair(p0, p1, v2);
      w[e] = pack_bf16(p0, p1);
    }
    tc::tmem_st16(s_col + 16 * cc, w);  // S columns 32 cc.. were read before P 16 cc.. is written
  }
  Redone r;
  r.m = m_new;
  r.l = l + sum_f32x2(ls[0]) + sum_f32x2(ls[1]);
  return r;
}

// The warp's 32 output rows (orow: this lane's; bit r of write: row r exists) from tensor memory:
// w0 O_k, plus w1 O_1 where both groups worked for the row, as bf16 or fp32.  64 bytes of every row
// at a time go through shared memory, so that a store instruction covers 8 rows x 64 bytes instead
// of 16 bytes of 32 rows.
template <int D>
__device__ __noinline__ void store_rows(uint32_t o_col, bool has0, bool has1, float w0, bool some0, float w1, bool some1,
                                        unsigned write, int64_t orow, void* out, bool bf16, uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const int row_bytes = bf16 ? D * 2 : D * 4;
  uint8_t* to[4];  // this lane's stores: 16 bytes of rows lane / 4 + 8 i
#pragma unroll
  for (int i = 0; i < 4; ++i)
    to[i] = static_cast<uint8_t*>(out) + __shfl_sync(0xffffffffu, orow, 8 * i + (lane >> 2)) * row_bytes + (lane & 3) * 16;
  // piece q of row r lies at q ^ ((r >> 1) & 3): no bank serves two rows at once
  const uint32_t at_w = stage + lane * 64, swz_w = (lane >> 1) & 3;
  const uint32_t at_r = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
  auto put = [&](const uint32_t* w, int off) {
#pragma unroll
    for (int q = 0; q < 4; ++q) st_shared_v4(at_w + ((q ^ swz_w) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = ld_shared_v4(at_r + 512 * i);
      if ((write >> (8 * i + (lane >> 2))) & 1u) *reinterpret_cast<uint4*>(to[i] + off) = u;
    }
    __syncwarp();
  };
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t x[2][16], w[16];
    if (has0) {
      tc::tmem_ld16(o_col + c, x[0]);
      tc::tmem_ld16(o_col + c + 16, x[1]);
    }
    if (has1) {
      uint32_t y[2][16];
      tc::tmem_ld16(o_col + 128 + c, y[0]);
      tc::tmem_ld16(o_col + 128 + c + 16, y[1]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float v = some0 ? __uint_as_float(x[e >> 4][e & 15]) * w0 : 0.f;
        if (some1) v = fmaf(__uint_as_float(y[e >> 4][e & 15]), w1, v);
        x[e >> 4][e & 15] = __float_as_uint(v);
      }
    } else {
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        x[e >> 4][e & 15] = some0 ? __float_as_uint(__uint_as_float(x[e >> 4][e & 15]) * w0) : 0u;
    }
    if (bf16) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        w[e] = pack_bf16(__uint_as_float(x[e >> 3][(2 * e) & 15]), __uint_as_float(x[e >> 3][(2 * e + 1) & 15]));
      put(w, 2 * c);
    } else {
      put(x[0], 4 * c);
      put(x[1], 4 * c + 64);
    }
  }
}

// One item after the other through all the roles: a role that is done with an item goes on to
// the next, so that loads and first scores of one item run under the epilogue of the one before.
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    chunk_tc_kernel(const __grid_constant__ PartialParams p, const __grid_constant__ CUtensorMap tmq,
                    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  constexpr int D = C::D, NST = C::NST, NB = C::NB;
  static_assert(sizeof(TcBars<C>) <= C::OFF_ML - C::OFF_BAR, "barriers");
  static_assert(2 * sizeof(TcItem) <= C::OFF_QS - C::OFF_ITEM, "items");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBars<C>* bars = reinterpret_cast<TcBars<C>*>(smem + C::OFF_BAR);
  TcItem* items = reinterpret_cast<TcItem*>(smem + C::OFF_ITEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.ck.G, Gr = p.ck.group_rows, gr_bits = 31 - __clz(Gr);  // (Gr is a power of two)

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], C::READERS);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_full[s], kRowsTile);
      mbar_init(&bars->pv_done[s], 1);
    }
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], C::FP8 ? 128 : 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->v8_full[s], 1);
      mbar_init(&bars->v8_empty[s], 128);
    }
    mbar_init(&bars->q8_full[0], 128);
    mbar_init(&bars->q8_full[1], 128);
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&bars->sc_full[s], 1);
    mbar_init(&bars->ml_full, kRowsTile);
    mbar_init(&bars->o1_free, kRowsTile);
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

  // Item r of this CTA has come (false: there is none, or a wait gave up) / is no longer read by
  // this warp.  The whole warp calls them.
  auto item_here = [&](int r) -> bool {
    const int s = r & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->item_full[s], (r >> 1) & 1, p.err, kDevErrFullWait))) return false;
    return items[s].it.b >= 0;
  };
  auto item_done = [&](int r) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[r & 1]);
  };
  auto next_item = [&](int r, TcItem* out) -> bool {
    if (!item_here(r)) return false;
    *out = items[r & 1];
    item_done(r);
    return true;
  };

  // fp8: the launch's 512 threads x 128 registers as 128 x (88 + 72 + 176 + 176)
  if (warp < 4) {
    if constexpr (C::FP8)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 3) {
      // ------------------------------------------------------------ scheduler
      // Items are handed out one by one (a counter that the plan kernel cleared), so that CTAs
      // with light items take more; one item ahead of the other roles.
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written
      const int total = __ldcg(p.ck.plan + kPlanItems);
      for (int r = 0;; ++r) {
        const int s = r & 1;
        if (r >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bars->item_empty[s], ((r >> 1) - 1) & 1, p.err, kDevErrEmptyWait)))
          break;
        int idx = blockIdx.x;
        if (r > 0) {
          if (lane == 0) idx = static_cast<int>(gridDim.x) + atomicAdd(p.ck.plan + kPlanNext, 1);
          idx = __shfl_sync(0xffffffffu, idx, 0);
        }
        TcItem t;
        t.it.b = -1;
        if (idx < total) {
          t.it = chunk_item_at(p.ck, idx);
          t.m0 = t.it.mt * 2 * kRowsTile;
          const int m_last = min(t.m0 + 2 * kRowsTile, t.it.n * Gr) - 1;
          t.pair = m_last - t.m0 >= kRowsTile ? 1 : 0;
          const int pos0 = t.it.m - t.it.n;
          t.tl = chunk_tiles(p.ck.window, p.ck.n_sink, p.ck.cap, pos0 + (t.m0 >> gr_bits), pos0 + (m_last >> gr_bits));
          const int tiles = (t.tl.n + 1) / 2, per = (tiles + t.it.n_chunk - 1) / t.it.n_chunk;
          const int i0 = min(t.it.c * per, tiles);
          t.h0 = 2 * i0;
          t.n_tiles = min(per, tiles - i0);
        }
        if (lane == 0) {
          items[s] = t;
          mbar_arrive(&bars->item_full[s]);
        }
        __syncwarp();
        if (t.it.b < 0) break;
      }
    } else if (warp != 1) {
      // ------------------------------------------------------------ TMA producers: 0 Q and K, 2 V
      // A warp each, so that neither waits for the other's ring; the pages and rows of the next
      // tile (four integer divisions and two dependent loads) are looked up behind this tile's
      // copies, not between a freed stage and its refill, which bounds a two-stage ring.
      const bool is_k = warp == 0;
      const CUtensorMap* map = is_k ? &tmk : &tmv;
      // (fp8: K codes go to the products as they are, V codes to a ring of their own, from which
      // the converter warps fill V's)
      uint64_t* full = is_k ? bars->k_full : C::FP8 ? bars->v8_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : C::FP8 ? bars->v8_empty : bars->v_empty;
      uint8_t* ring = smem + (is_k ? C::OFF_K : C::FP8 ? C::OFF_V8 : C::OFF_V);
      if (tc::elect_one()) {
        tma_prefetch_desc(map);
        if (is_k) tma_prefetch_desc(&tmq);
      }
      __syncwarp();
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err, kDevErrEmptyWait));
      };
      TcItem t;
      int done = 0, nq = 0;  // tiles and query tiles loaded so far
      bool ok = true;
      for (int r = 0; ok && next_item(r, &t); ++r) {
        if (t.n_tiles == 0) continue;
        int page[2], at[2];  // of a tile's two halves
        float scale = 0.f;   // fp8: lanes 0-3 of the K loader
        auto look_up = [&](int i) {
          const int first[2] = {t.token(2 * i), t.token(2 * i + 1)};
          // a second half at or past the capacity holds no token: it takes the first one's page
          // instead of an entry behind the table's row
          const int a = first[0], b = first[1] < p.ck.cap ? first[1] : a;
          at[0] = a % p.block_len;
          at[1] = b % p.block_len;
          page[0] = kv_page_of(p, t.it.b, a);
          page[1] = kv_page_of(p, t.it.b, b);
          if constexpr (C::FP8) {
            // the scales of both halves, a lane each (K, V, K, V).  Halves in which no row sees a token,
            // and pages outside the cache, take 0: their scales may be anything
            const int hf = (lane >> 1) & 1, tok = first[hf], pg = page[hf];
            const bool seen = (tok < t.tl.hi && tok + kHalf > t.tl.lo) || tok < t.tl.sinks;
            scale = 0.f;
            if (is_k && lane < 4 && seen && pg >= 0 && pg < p.num_blocks) {
              const int per = p.block_len / p.scale_block;
              const int64_t x = (static_cast<int64_t>(pg) * p.Hkv + t.it.g) * per + at[hf] / p.scale_block;
              scale = __ldg(((lane & 1) ? p.v_scale : p.k_scale) + x);
            }
          }
        };
        look_up(0);
        if (is_k) {
          // the item before has no scores left to compute
          if (nq > 0 && !wait_all(&bars->q_empty, (nq - 1) & 1)) break;
          if (tc::elect_one()) {
            mbar_arrive_expect_tx(&bars->q_full, (1 + t.pair) * C::TILE);
            for (int k = 0; k <= t.pair; ++k)
              for (int bx = 0; bx < NB; ++bx)
                tma_4d(smem + k * C::TILE + bx * C::BOX, &tmq, &bars->q_full, bx * 64, t.it.g * G,
                       t.it.row0 + ((t.m0 + k * kRowsTile) >> gr_bits), 0);
          }
          __syncwarp();
          ++nq;
        }
        for (int i = 0; i < t.n_tiles; ++i) {
          const int s = done % NST;
          ok = done < NST || wait_all(&empty[s], ((done / NST) - 1) & 1);
          if (!ok) break;
          if (tc::elect_one()) {
            mbar_arrive_expect_tx(&full[s], C::LOAD);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int bx = 0; bx < C::LOAD_BOXES; ++bx)
                tma_4d(ring + s * C::LOAD + bx * C::BOX + hf * (C::BOX / 2), map, &full[s], bx * C::LOAD_BOX_ELEMS, at[hf],
                       t.it.g, page[hf]);
          }
          __syncwarp();
          if constexpr (C::FP8) {
            if (is_k) {
              // slot of tile x again at x + 8: its codes take a stage that the scores of x + 8 - NST left,
              // which were issued after P V of x: the softmax of x is done
              const int sl = done % kScaleSlots;
              if (lane < 4) reinterpret_cast<float*>(&bars->scales[sl])[lane] = scale;
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->sc_full[sl]);
            }
          }
          ++done;
          if (i + 1 < t.n_tiles) look_up(i + 1);
        }
      }
      // every issued copy lands before the CTA may exit
      for (int i = max(0, done - NST); i < done; ++i)
        if (!mbar_wait(&full[i % NST], (i / NST) & 1, p.err, kDevErrDrainWait)) break;
      if (is_k && nq > 0) mbar_wait(&bars->q_full, (nq - 1) & 1, p.err, kDevErrDrainWait);
    } else {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp waits, one elected lane issues; a tile's stage is a compile-time constant,
      // so every operand is a constant offset.
      // (format 0 of kind::f8f6f4 is e4m3, as 0 of kind::f16 is fp16)
      const uint32_t idesc_s = tc::idesc_f16(128, kTN, !C::FP8, false, false);
      const uint32_t idesc_pv = tc::idesc_f16(128, D, true, false, true);
      const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
      const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), C::BOX, 1024);
      // A descriptor at a constant offset, by one 32-bit addition where it is used: kept as they are
      // over the loops, the 64-bit sums of every product take more registers than the warp has (the
      // address field ends in the low word, shared memory ends below its 18 bits)
      auto low_of = [](uint64_t d) -> uint32_t {
        uint32_t lo = static_cast<uint32_t>(d);
        asm volatile("" : "+r"(lo));
        return lo;
      };
      auto at = [](uint64_t d, uint32_t lo, uint32_t bytes) -> uint64_t {
        return (d & 0xFFFFFFFF00000000ull) | (lo + (bytes >> 4));
      };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err, kDevErrFullWait));
      };
      auto issue_s = [&](int k, int q, int stage) {  // S_k = Q_q K^T
        const uint32_t ql = low_of(qd), kl = low_of(kd);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t in_box = (ks >> 2) * C::BOX + (ks & 3) * 32;
          const uint64_t qa = at(qd, ql, q * C::TILE + in_box);
          if constexpr (C::FP8)  // the large parts of Q over 4 steps of 32 codes, then the small ones
            tc::mma_f8_ss(tmem + kColS + 128 * k, qa, at(kd, kl, stage * C::LOAD + (ks & 3) * 32), idesc_s, ks > 0 ? 1u : 0u);
          else
            tc::mma_f16_ss(tmem + kColS + 128 * k, qa, at(kd, kl, stage * C::LOAD + in_box), idesc_s, ks > 0 ? 1u : 0u);
        }
        tc::mma_commit(smem_u32(&bars->s_full[k]));
      };
      auto issue_pv = [&](int k, int stage, uint32_t acc0) {  // O_k += P_k V
        const uint32_t vl = low_of(vd);
#pragma unroll
        for (int ks = 0; ks < kTN / 16; ++ks)
          tc::mma_f16_ts(tmem + kColO + 128 * k, tmem + kColS + 128 * k + ks * 8, at(vd, vl, stage * C::TILE + ks * 2048),
                         idesc_pv, ks > 0 ? 1u : acc0);
        tc::mma_commit(smem_u32(&bars->pv_done[k]));
      };
      // runs fn with tile number x's stage as a constant
      auto at_stage = [&](int x, auto&& fn) {
        const int s = x % NST;
        if (s == 0) fn(Int<0>{});
        if (s == 1) fn(Int<1>{});
        if constexpr (NST == 4) {
          if (s == 2) fn(Int<2>{});
          if (s == 3) fn(Int<3>{});
        }
      };
      TcItem t;
      int base = 0, nq = 0;          // tiles and query tiles of the items before
      uint32_t np[2] = {0u, 0u};     // tiles of each softmax group so far
      bool ok = true;
      for (int r = 0; ok && next_item(r, &t); ++r) {
        const int n = t.n_tiles;
        if (n == 0) continue;
        ok = C::FP8 ? wait_all(&bars->q8_full[nq & 1], (nq >> 1) & 1) : wait_all(&bars->q_full, nq & 1);
        if (!ok) break;
        ++nq;
        // scores of tile x (both groups, or group x & 1 in solo mode); the last ones free Q
        if (t.pair) {
          // tile i: PV0(i), S0(i+1), PV1(i), S1(i+1)
          ok = wait_all(&bars->k_full[base % NST], (base / NST) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          at_stage(base, [&](auto st) {
            constexpr int ST = decltype(st)::value;
            if (tc::elect_one()) {
              issue_s(0, 0, ST);
              issue_s(1, 1, ST);
              tc::mma_commit(smem_u32(&bars->k_empty[ST]));
              if (n == 1) tc::mma_commit(smem_u32(&bars->q_empty));
            }
            __syncwarp();
          });
          auto tile = [&](auto st, int i) {
            constexpr int ST = decltype(st)::value, NX = (ST + 1) % NST;
            const int x = base + i;
            const bool more = i + 1 < n;
            // tiles first, the softmax last: a wait costs 100 cycles and more even for what is there
            ok = wait_all(&bars->v_full[ST], (x / NST) & 1) && (!more || wait_all(&bars->k_full[NX], ((x + 1) / NST) & 1)) &&
                 wait_all(&bars->p_full[0], np[0] & 1);
            if (!ok) return;
            ++np[0];
            tc::fence_after_sync();
            if (tc::elect_one()) {
              issue_pv(0, ST, i > 0 ? 1u : 0u);
              if (more) issue_s(0, 0, NX);
            }
            __syncwarp();
            ok = wait_all(&bars->p_full[1], np[1] & 1);
            if (!ok) return;
            ++np[1];
            tc::fence_after_sync();
            if (tc::elect_one()) {
              issue_pv(1, ST, i > 0 ? 1u : 0u);
              tc::mma_commit(smem_u32(&bars->v_empty[ST]));
              if (more) {
                issue_s(1, 1, NX);
                tc::mma_commit(smem_u32(&bars->k_empty[NX]));
                if (i + 2 == n) tc::mma_commit(smem_u32(&bars->q_empty));
              }
            }
            __syncwarp();
          };
          // unrolled by the ring depth, entered at the stage that the items before left
          int i = 0;
          const int enter = base % NST;
          for (bool first = true; ok && i < n; first = false) {
            if (!first || enter <= 0) {
              tile(Int<0>{}, i);
              if (!ok || ++i >= n) break;
            }
            if (!first || enter <= 1) {
              tile(Int<1>{}, i);
              if (!ok || ++i >= n) break;
            }
            if constexpr (NST == 4) {
              if (!first || enter <= 2) {
                tile(Int<2>{}, i);
                if (!ok || ++i >= n) break;
              }
              tile(Int<3>{}, i);
              ++i;
            }
          }
        } else {
          // tile i belongs to group i & 1: PV(i), then S(i + 2)
          auto scores = [&](int i) {
            at_stage(base + i, [&](auto st) {
              constexpr int ST = decltype(st)::value;
              ok = wait_all(&bars->k_full[ST], ((base + i) / NST) & 1);
              if (!ok) return;
              tc::fence_after_sync();
              if (tc::elect_one()) {
                if (i & 1)
                  issue_s(1, 0, ST);
                else
                  issue_s(0, 0, ST);
                tc::mma_commit(smem_u32(&bars->k_empty[ST]));
                if (i + 1 == n) tc::mma_commit(smem_u32(&bars->q_empty));
              }
              __syncwarp();
            });
          };
          scores(0);
          if (ok && n > 1) scores(1);
          for (int i = 0; i < n && ok; ++i) {
            at_stage(base + i, [&](auto st) {
              constexpr int ST = decltype(st)::value;
              const int k = i & 1;
              ok = wait_all(&bars->p_full[k], np[k] & 1) && wait_all(&bars->v_full[ST], ((base + i) / NST) & 1);
              if (!ok) return;
              ++np[k];
              tc::fence_after_sync();
              if (tc::elect_one()) {
                if (k)
                  issue_pv(1, ST, i > 1 ? 1u : 0u);
                else
                  issue_pv(0, ST, i > 1 ? 1u : 0u);
                tc::mma_commit(smem_u32(&bars->v_empty[ST]));
              }
              __syncwarp();
            });
            if (ok && i + 2 < n) scores(i + 2);
          }
        }
        base += n;
      }
    }
  } else if (warp >= 12) {  // (fp8 only: no such warps otherwise)
    // ------------------------------------------------------------ fp8: Q split, V codes to bf16
    if constexpr (C::FP8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      const int row = (warp - 12) * 32 + lane;
      // Q for the products with e4m3 keys: a row times the power of two that puts its largest
      // magnitude in [2^7, 2^8) is the sum of two e4m3 values, the rounded one and the rest.  A bf16
      // value's 8 bits are 4 and 4, so the sum is exact down to 2^-9 of the row's largest and off
      // by 2^-17 of it at most below (half the subnormal step, 2^-10, against 2^7).  The rounded parts (128 bytes) go over the row's first 64
      // values, the rests over its last 64, each after what it overwrites was read.
      auto split_q = [&](uint8_t* q) -> float {
        auto chunk = [&](int c) {
          return reinterpret_cast<uint4*>(q + (c >> 3) * C::BOX + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        };
        uint32_t most = 0u;  // magnitudes order as their bits; a NaN is above infinity
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          const uint4 u = *chunk(c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) most = max(most, max((w[j] << 16) & 0x7FFF0000u, w[j] & 0x7FFF0000u));
        }
        const bool finite = most < 0x7F800000u;
        const int e = most == 0u ? 0 : min(max(static_cast<int>(most >> 23) - 127 - 7, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        // a pair's codes: the rounded values in the low halves of hi, the rests' in those of lo
        auto split = [&](uint32_t w, uint32_t& hi, uint32_t& lo) {
          const float x = bf16_lo(w) * down, y = bf16_hi(w) * down;
          const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
          const uint32_t back = e4m3x2_to_f16x2(h);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
          hi = h;
          lo = __nv_cvt_float2_to_fp8x2(make_float2(x - f.x, y - f.y), __NV_SATFINITE, __NV_E4M3);
        };
        auto split_chunk = [&](const uint4& u, uint32_t* hi, uint32_t* lo) {  // 8 values: 2 words each
          uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
          split(u.x, h0, l0);
          split(u.y, h1, l1);
          split(u.z, h2, l2);
          split(u.w, h3, l3);
          hi[0] = h0 | (h1 << 16), hi[1] = h2 | (h3 << 16);
          lo[0] = l0 | (l1 << 16), lo[1] = l2 | (l3 << 16);
        };
        uint32_t lo[16];  // the rests of the values read so far and not yet written
#pragma unroll
        for (int c = 0; c < 8; c += 2) {  // first 64 values
          uint32_t hi[4];
          const uint4 u = *chunk(c), v = *chunk(c + 1);
          split_chunk(u, hi, lo + 2 * c);
          split_chunk(v, hi + 2, lo + 2 * c + 2);
          *chunk(c / 2) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
#pragma unroll
        for (int c = 0; c < 8; c += 4) {  // last 64, four chunks read before two of them are written
          uint32_t hi[8], rest[8];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint4 u = *chunk(8 + c + d);
            split_chunk(u, hi + 2 * d, rest + 2 * d);
          }
          *chunk(4 + c / 2) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *chunk(5 + c / 2) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
          if (c == 0) {  // chunks 8 .. 11 are read: the first values' rests; these rests wait in their place
#pragma unroll
            for (int d = 0; d < 4; ++d) *chunk(8 + d) = make_uint4(lo[4 * d], lo[4 * d + 1], lo[4 * d + 2], lo[4 * d + 3]);
#pragma unroll
            for (int d = 0; d < 8; ++d) lo[d] = rest[d];
          } else {  // chunks 12 .. 15 are read
            *chunk(12) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *chunk(13) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
            *chunk(14) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            *chunk(15) = make_uint4(rest[4], rest[5], rest[6], rest[7]);
          }
        }
        // an infinity or a NaN in the row makes its scores NaN
        return finite ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __int_as_float(0x7fc00000);
      };
      // One thread a token row: 16 codes of a 16-byte chunk become the 32 bytes of two chunks of
      // the 128-byte-swizzled bf16 tile (both sides conflict-free: eight rows, eight chunks).
      auto convert = [&](const uint8_t* from, uint8_t* to) {
        uint32_t odd = 0u;  // bit 7 of a byte: a NaN code among the row's
#pragma unroll 4
        for (int c = 0; c < 8; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(from + row * 128 + ((c ^ (row & 7)) << 4));
          uint8_t* d = to + (c >> 2) * C::BOX + row * 128;
          const int d0 = 2 * (c & 3);
          uint4 lo, hi;
          e4m3x4_to_bf16(u.x, lo.x, lo.y, odd);
          e4m3x4_to_bf16(u.y, lo.z, lo.w, odd);
          e4m3x4_to_bf16(u.z, hi.x, hi.y, odd);
          e4m3x4_to_bf16(u.w, hi.z, hi.w, odd);
          *reinterpret_cast<uint4*>(d + ((d0 ^ (row & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(d + (((d0 + 1) ^ (row & 7)) << 4)) = hi;
        }
        if (odd & 0x80808080u) {  // rare: put the NaNs in
          for (int x = 0; x < 128; ++x) {
            const uint8_t code = from[row * 128 + (((x >> 4) ^ (row & 7)) << 4) + (x & 15)];
            if ((code & 0x7Fu) == 0x7Fu) {
              const int b = 2 * (x & 63);
              *reinterpret_cast<uint16_t*>(to + (x >> 6) * C::BOX + row * 128 + (((b >> 4) ^ (row & 7)) << 4) + (b & 15)) =
                  0x7FC0u;
            }
          }
        }
      };
      int done = 0, nq = 0;  // tiles and query tiles so far
      bool ok = true;
      for (int r = 0; ok && item_here(r); ++r) {
        const int n = items[r & 1].n_tiles, pair = items[r & 1].pair;
        item_done(r);
        if (n == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full, nq & 1, p.err, kDevErrFullWait));
        if (!ok) break;
        float* qs = reinterpret_cast<float*>(smem + C::OFF_QS) + (nq & 1) * 2 * kRowsTile;
        for (int k = 0; k <= pair; ++k) qs[k * kRowsTile + row] = split_q(smem + k * C::TILE);
        fence_proxy_async_smem();
        mbar_arrive(&bars->q8_full[nq & 1]);
        ++nq;
        for (int i = 0; i < n && ok; ++i, ++done) {
          const int s = done % NST;
          ok = mbar_wait(&bars->v8_full[s], (done / NST) & 1, p.err, kDevErrFullWait) &&
               (done < NST || mbar_wait(&bars->v_empty[s], ((done / NST) - 1) & 1, p.err, kDevErrEmptyWait));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          convert(smem + C::OFF_V8 + s * C::LOAD, smem + C::OFF_V + s * C::TILE);
          fence_proxy_async_smem();
          mbar_arrive(&bars->v_full[s]);
          mbar_arrive(&bars->v8_empty[s]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    if constexpr (C::FP8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int k = (warp - 4) >> 2;
    const int lgrp = warp & 3;         // TMEM lane group of this warp
    const int row = lgrp * 32 + lane;  // row inside the query tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lgrp * 32) << 16);
    const uint32_t s_col = t_lane + kColS + 128 * k;
    const uint32_t o_col = t_lane + kColO + 128 * k;
    float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
    int4* mine = reinterpret_cast<int4*>(smem + C::OFF_ROW) + k * kRowsTile + row;
    int base = 0;              // tiles of the items before
    uint32_t np = 0, np1 = 0;  // tiles of this group, and of group 1, so far
    uint32_t n_solo = 0, nq = 0;  // solo items, items with tiles so far
    WarpWait wait(p.err);
    for (int r = 0; wait.ok && item_here(r); ++r) {
      const TcItem& t = items[r & 1];  // read in place: registers are short here
      const bool pair = t.pair != 0;
      // What only edge tiles and the epilogue need waits in shared memory: the registers are full
      // of scores and weights.
      bool active;                  // some row of this warp exists
      int hi_min, lo_max, sink_min;  // a tile in [lo_max, hi_min) (or below sink_min) every row sees
      {
        const int m = t.m0 + (pair ? k * kRowsTile : 0) + row;
        const int t_q = m >> gr_bits, hg = m & (Gr - 1);
        const bool valid = m < t.it.n * Gr && hg < G;
        const int pos = t.it.m - t.it.n + t_q;
        // visible tokens of this row: [lo_row, hi_row) and [0, sink_row)
        const int hi_row = valid ? min(max(pos + 1, 0), p.ck.cap) : 0;
        const int lo_row = (valid && p.ck.window > 0 && pos >= p.ck.window) ? pos - p.ck.window + 1 : 0;
        const int sink_row = min(p.ck.n_sink, hi_row);
        active = __any_sync(0xffffffffu, valid);
        hi_min = __reduce_min_sync(0xffffffffu, valid ? hi_row : INT_MAX);
        lo_max = __reduce_max_sync(0xffffffffu, lo_row);
        sink_min = __reduce_min_sync(0xffffffffu, valid ? sink_row : INT_MAX);
        *mine = make_int4(hi_row, lo_row, sink_row, valid ? 1 : 0);
      }
      float m_used = -INFINITY, l_sum = 0.f;
      float q_scale = 0.f;  // fp8: the score scale times the row's own
      const int step = pair ? 1 : 2;  // this group's tiles: all, or every other

      int j = 0;  // tiles of the item done
      for (int i = pair ? 0 : k; i < t.n_tiles; i += step, ++j) {
        const int ta = t.token(2 * i), tb = t.token(2 * i + 1);  // the halves' first tokens
        if (!wait(&bars->s_full[k], np & 1, kDevErrFullWait)) break;
        ++np;
        tc::fence_after_sync();
        if (active) {
          auto all_see = [&](int a) { return hi_min >= a + kHalf && (lo_max <= a || sink_min >= a + kHalf); };
          const bool edge = !all_see(ta) || !all_see(tb);
          // score scale (base 2) and V scale of the tile's halves
          float sl[2] = {p.scale_log2, p.scale_log2}, vs[2] = {1.f, 1.f};
          if constexpr (C::FP8) {
            const int x = base + i;
            if (!wait(&bars->sc_full[x % kScaleSlots], (x / kScaleSlots) & 1, kDevErrFullWait)) break;
            const float4 sc = bars->scales[x % kScaleSlots];
            if (j == 0) {
              // the row's own scale.  (Q of the item after the next one is split only after the
              // next one's last scores, which follow this item's last P V)
              if (!wait(&bars->q8_full[nq & 1], (nq >> 1) & 1, kDevErrFullWait)) break;
              q_scale = p.scale_log2 *
                        reinterpret_cast<const float*>(smem + C::OFF_QS)[((nq & 1) * 2 + (pair ? k : 0)) * kRowsTile + row];
            }
            sl[0] = q_scale * sc.x, vs[0] = sc.y, sl[1] = q_scale * sc.z, vs[1] = sc.w;
          }
          if constexpr (C::FP8) {  // a masked score is an infinity that the scale makes -inf
            sl[0] = sl[0] == 0.f ? 1e-37f : sl[0];
            sl[1] = sl[1] == 0.f ? 1e-37f : sl[1];
          }
          if (edge) {
            const float inf = -INFINITY;  // after the scale
            hide_scores(s_col, ta, tb, *mine, hi_min, lo_max, sink_min, C::FP8 && sl[0] < 0.f ? -inf : inf,
                        C::FP8 && sl[1] < 0.f ? -inf : inf);
          }
          if (__any_sync(0xffffffffu, m_used == -INFINITY)) m_used = first_max<C::FP8>(s_col, m_used, sl[0], sl[1]);
          uint32_t pk[kTN / 2];
          uint64_t ls[2] = {0ull, 0ull};  // fp32 pair sums of p
          const float base0 = (m_used == -INFINITY) ? 0.f : m_used;
          {
#pragma unroll
            for (int cc = 0; cc < kTN / 32; ++cc) {
              uint32_t x[2][16];
              tc::tmem_ld16(s_col + 32 * cc, x[0]);
              tc::tmem_ld16(s_col + 32 * cc + 16, x[1]);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float a0, a1;
                fma_pair(__uint_as_float(x[e >> 3][(2 * e) & 15]), __uint_as_float(x[e >> 3][(2 * e + 1) & 15]),
                         sl[cc >> 1], -base0, a0, a1);
                float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
                ls[e & 1] = add_f32x2(ls[e & 1], p0, p1);
                if constexpr (C::FP8) mul_pair(p0, p1, vs[cc >> 1]);  // V = code * scale
                pk[16 * cc + e] = pack_bf16(p0, p1);
              }
            }
          }
          const bool need = !(sum_f32x2(ls[0]) + sum_f32x2(ls[1]) <= kTileSumLimit) || fabsf(base0) > kLargeScore;
          if (__any_sync(0xffffffffu, need)) {
            const Redone again = redo_tile<D, C::FP8>(s_col, o_col, need, m_used, l_sum, sl[0], sl[1], vs[0], vs[1]);
            m_used = again.m;
            l_sum = again.l;
          } else {
            l_sum += sum_f32x2(ls[0]) + sum_f32x2(ls[1]);
#pragma unroll
            for (int cc = 0; cc < kTN / 32; ++cc) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = pk[16 * cc + e];
              tc::tmem_st16(s_col + 16 * cc, w);
            }
          }
          tc::tmem_wait_st();
        }
        auto inside = [&](int a) { return (a >= t.tl.lo && a + kHalf <= t.tl.hi) || a + kHalf <= t.tl.sinks; };
        if ((k == 0 || !pair) && !(inside(ta) && inside(tb))) {
          // tokens that no row of the item sees may hold anything: zero their V rows, so that
          // p = 0 really counts nothing
          const int x = base + i, s = x % NST;
          if (!wait(&bars->v_full[s], (x / NST) & 1, kDevErrFullWait)) break;
          for (int y = row >> 3; y < kTN; y += 16) {  // 8 threads a row
            const int tok = y < kHalf ? ta + y : tb + y - kHalf;
            if (!((tok >= t.tl.lo && tok < t.tl.hi) || tok < t.tl.sinks)) {
              uint8_t* vt = smem + C::OFF_V + s * C::TILE + y * 128 + (row & 7) * 16;
              for (int bx = 0; bx < NB; ++bx) *reinterpret_cast<uint4*>(vt + bx * C::BOX) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        mbar_arrive(&bars->p_full[k]);
      }
      base += t.n_tiles;
      if (t.n_tiles > 0) ++nq;
      const int tiles1 = pair ? t.n_tiles : t.n_tiles / 2;  // group 1's
      np1 += tiles1;
      if (!wait.ok) break;

      // ---- epilogue: O / l and lse
      // solo: the two groups' weights.  A group that summed nothing has l = 0 (its O may be
      // anything); a NaN among the scores keeps l NaN, and the row is NaN
      float a0 = 1.f, a1 = 0.f;
      bool some0 = l_sum != 0.f, some1 = false;
      if (!pair) {
        if (k == 1) {
          ml[2 * row] = m_used;
          ml[2 * row + 1] = l_sum;
          mbar_arrive(&bars->ml_full);
          // O1 and (m, l) are read before the next item changes them
          if (!wait(&bars->o1_free, n_solo & 1, kDevErrEmptyWait)) break;
          ++n_solo;
          tc::fence_after_sync();
          item_done(r);
          continue;
        }
        if (!wait(&bars->ml_full, n_solo & 1, kDevErrFullWait)) break;
        ++n_solo;
        const float m1 = ml[2 * row], l1 = ml[2 * row + 1];
        const float mm = fmaxf(m_used, m1);
        some1 = l1 != 0.f;
        a0 = some0 ? fast_exp2(m_used - mm) : 0.f;
        a1 = some1 ? fast_exp2(m1 - mm) : 0.f;
        l_sum = (some0 ? a0 * l_sum : 0.f) + (some1 ? a1 * l1 : 0.f);
        m_used = mm;
      }
      if (j > 0 && !wait(&bars->pv_done[k], (np - 1) & 1, kDevErrFullWait)) break;
      const bool both = !pair && tiles1 > 0;
      if (both && !wait(&bars->pv_done[1], (np1 - 1) & 1, kDevErrFullWait)) break;
      tc::fence_after_sync();
      const bool some = some0 || some1;
      const float inv = some ? 1.f / l_sum : 0.f;
      a0 *= inv;
      a1 *= inv;
      constexpr float kLn2 = 0.6931471805599453f;
      const float lse = some ? (m_used + __log2f(l_sum)) * kLn2 : -INFINITY;
      const bool direct = t.it.n_chunk == 1;
      const bool valid = mine->w != 0;
      const int m = t.m0 + (pair ? k * kRowsTile : 0) + row;
      const int t_q = m >> gr_bits, h = t.it.g * G + (m & (Gr - 1));
      const int64_t orow = direct ? (static_cast<int64_t>(t.it.row0) + t_q) * p.Hq + h
                                  : t.it.part_row + (static_cast<int64_t>(t.it.c) * t.it.n + t_q) * p.Hq + h;
      // an empty partial's o is never read
      const unsigned write_o = __ballot_sync(0xffffffffu, valid && (direct || some));
      if (write_o != 0u) {
        store_rows<D>(o_col, t.n_tiles > 0, both, some0 ? a0 : 0.f, some0, some1 ? a1 : 0.f, some1, write_o, orow,
                      direct ? p.ck.out : p.out_o, direct, smem_u32(smem + C::OFF_OUT + (warp - 4) * (32 * 64)));
      }
      if (valid) (direct ? p.ck.lse : p.out_lse)[orow] = lse;
      // (the next tile's p_full arrival orders these TMEM reads before the next PV writes O)
      tc::fence_before_sync();
      if (!pair) mbar_arrive(&bars->o1_free);
      item_done(r);
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
  // a programmatic dependent of the plan kernel: its CTAs set themselves up meanwhile
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(std::min<int64_t>(n_items, p.ck.n_wave)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_tc_kernel<C>, p, tmq, tmk, tmv);
}

}  // namespace

int chunk_tc_rows() { return 2 * kRowsTile; }
int chunk_tc_kv_tile() { return kTN; }
int chunk_tc_kv_box() { return kHalf; }

cudaError_t launch_chunk_tc(const PartialParams& p, int32_t d, bool fp8, const CUtensorMap& tmq, const CUtensorMap& tmk,
                            const CUtensorMap& tmv, int64_t n_items, cudaStream_t stream) {
  if (fp8) return launch_cfg<TcCfg<128, true>>(p, tmq, tmk, tmv, n_items, stream);
  if (d == 64) return launch_cfg<TcCfg<64, false>>(p, tmq, tmk, tmv, n_items, stream);
  return launch_cfg<TcCfg<128, false>>(p, tmq, tmk, tmv, n_items, stream);
}

}  // namespace skv
