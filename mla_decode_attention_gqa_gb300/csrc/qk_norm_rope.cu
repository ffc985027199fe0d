// Norm of every query and key head, position rotation, and the write into the paged cache, in
// one pass over the new tokens (qk_norm_rope_append).
//
// For each token and head x in R^d:   y = x w / sqrt(mean(x^2) + eps)   (queries and keys),
//   (y_a, y_b) <- (y_a cos_j - y_b sin_j, y_b cos_j + y_a sin_j)   for j < rot / 2, with
//   (a, b) = (j, j + rot/2), or (2j, 2j + 1) interleaved; cos_j, sin_j: the row of the token's
//   position in the caller's tables.  The query goes out in bf16, the key to its page row in
//   bf16, as the e4m3 code of y / scale (the block scale that the cache holds), or as 4-bit codes
//   with scales made here (see store_fp4), the value likewise without norm and rotation.
//   Everything between the loads and the one rounding at the store is in fp32.
//
// Bound by HBM: each input is read once and each output written once.  A warp copies the heads by
// bulk copies into a ring, 32 heads a stage, so that 40 KB a CTA are on their way whatever the
// others wait for (heads loaded to registers ahead of their use: 68 us for 4096 tokens of
// 128 + 16 heads, this way 54: 5.7 TB/s of the 6.8 that a copy reaches).  8 lanes take one head, as
// two chunks of d / 16 values that the rotation pairs, so that it needs no exchange between lanes,
// the sum of squares is three shuffles for four heads, and the arithmetic runs on packed pairs.
// The chains token -> sequence -> position -> page and table row of all tokens of a CTA's run go
// side by side, a lane each, under the first copies, and leave the run's rotations and scales in
// shared memory (looked up by each head's lanes at a new token: 58 us).
#include <cuda_runtime.h>

#include <algorithm>

#include "skv_common.cuh"
#include "skv_internal.h"

namespace skv {

namespace {

constexpr int kWarps = 8;              // consumer warps
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kGroups = kWarps * 4;    // heads of a stage
constexpr int kStages = 5;             // 40 KB for heads of 128
// CTAs an SM.  bf16: two, a token's rotation held in registers while its heads pass (4096 tokens of
// 128 + 16 heads 54 us; three CTAs that read it from shared memory for each head 56).  fp8: three,
// whose warps hide the conversions (6800 tokens of 64 + 16 heads 62 us against 70).  4-bit: three as well (8192
// tokens of 64 + 16 heads 73 us, 0.64 of the measured copy rate, against 75; the instructions of the key and value
// heads, 16 divisions a lane among them, which products with a reciprocal would do in 4 us less, but on the
// wrong side of a middle between two codes).
constexpr int ctas_per_sm(PageFormat pages) { return pages == kPagesBf16 ? 2 : 3; }
constexpr int kMaxTokens = 64;         // tokens a CTA's run may touch: 8 a warp
constexpr int kScaleHeads = 16;        // KV heads whose scales wait in shared memory

// ---- two fp32 values in one 64-bit register (packed round-to-nearest operations)
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t swap2(uint64_t v) {
  float x, y;
  unpack2(v, x, y);
  return pack2(y, x);
}

// Untiled bulk copy (16-byte aligned addresses, a multiple of 16 bytes) completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Arrival once `sum`, a sum of squares, is there.  One lane arrives for the loads of eight: behind them in the
// program alone, with neither a __syncwarp() nor a use of what they bring between, the arrival does not say that the
// other lanes' are done, and the next copy into the stage overtook some of them (in the first launch of a process, whose
// warps wait for their instructions, 5 of 90 had a head or two of the first stage read after its refill).
// The sum holds all values of the eight lanes.  It is tested against a value that it cannot have, so the arrival
// needs it, and it needs what was loaded.
__device__ __forceinline__ void arrive_after(uint64_t* bar, float sum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0x80000001;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(__float_as_uint(sum))
      : "memory");
}

// H bf16 values as packed words.
template <int H>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* p, uint32_t* w) {
  if constexpr (H == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}
template <int H>
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const uint32_t* w) {
  if constexpr (H == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// e4m3 codes of x / scale, saturated at +-448; a scale that is not a positive number stores
// zeros (the value that such a block stands for).  A product with the reciprocal where that is
// finite (off by 2^-23 of the quotient before the rounding to 2^-4), else a division.
template <int H>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const uint64_t* x, float scale) {
  const bool ok = scale > 0.f && scale <= 3.402823466e38f, tiny = scale < 1.1754944e-38f;
  const float inv = ok && !tiny ? __frcp_rn(scale) : 0.f;
  uint32_t w[H / 4];
#pragma unroll
  for (int i = 0; i < H / 4; ++i) {
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float u, v;
      unpack2(x[2 * i + j], u, v);
      float2 z = make_float2(u * inv, v * inv);
      if (ok && tiny) z = make_float2(__fdiv_rn(u, scale), __fdiv_rn(v, scale));
      if (!ok) z = make_float2(0.f, 0.f);
      codes |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3)) << (16 * j);
    }
    w[i] = codes;
  }
  if constexpr (H == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Where a head's chunk `id` (of H values) is: lane of its 8, and which of the lane's two chunks.
struct ChunkAt {
  int lane, second;
};
template <int H>
__device__ __forceinline__ ChunkAt chunk_at(int id, bool inter, int rot) {
  const int n = 16, half = inter ? 8 : rot / (2 * H), turned = inter ? n : rot / H, rest = (n - turned) / 2;
  ChunkAt c;
  if (id < turned) {
    c.second = id >= half;
    c.lane = c.second ? id - half : id;
  } else {
    c.second = id >= turned + rest;
    c.lane = id - turned - (c.second ? rest : 0) + half;
  }
  return c;
}

// One of a lane's chunks as 4-bit codes: 8 of the block's 16 dims, whose largest magnitude is `most`.
//   s = e4m3(most / (6 h)),  code = e2m1(y / (s h)),  h: the head's scale.
// The block's first chunk stores s.  A NaN in the block makes s NaN, and so the block; a magnitude
// past 2688 h saturates.
__device__ __forceinline__ void store_fp4(uint8_t* codes, uint8_t* scale, const uint64_t* x, float most, float h) {
  const uint32_t s = h > 0.f ? __nv_cvt_float_to_fp8(__fdiv_rn(most, 6.f * h), __NV_SATFINITE, __NV_E4M3) : 0u;
  const uint32_t wide = e4m3x2_to_f16x2(static_cast<uint16_t>(s));
  const float by = __low2float(*reinterpret_cast<const __half2*>(&wide)) * h;
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    unpack2(x[j], y[2 * j], y[2 * j + 1]);
    // (a division: values of few bits often lie just between two codes, where a product with the
    // reciprocal would fall to either side)
    y[2 * j] = __fdiv_rn(y[2 * j], by), y[2 * j + 1] = __fdiv_rn(y[2 * j + 1], by);
  }
  *reinterpret_cast<uint32_t*>(codes) = by > 0.f ? f32x8_to_e2m1x8(y) : 0u;
  if (scale) *scale = static_cast<uint8_t>(s);
}

// H norm weights as packed pairs.
template <int H>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int64_t at, uint64_t* x) {
  if (bf16) {
    uint32_t u[H / 2];
    load_chunk<H>(static_cast<const __nv_bfloat16*>(w) + at, u);
#pragma unroll
    for (int i = 0; i < H / 2; ++i) x[i] = pack2(bf16_lo(u[i]), bf16_hi(u[i]));
  } else {
#pragma unroll
    for (int i = 0; i < H; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at + i));
      x[i / 2] = pack2(u.x, u.y);
      x[i / 2 + 1] = pack2(u.z, u.w);
    }
  }
}

// Sequence of packed row `row`: the last b with cu_q[b] <= row, if row < cu_q[b + 1]; else -1.
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int row) {
  if (__ldg(cu_q) > row) return -1;
  int lo = 0;
  for (int n = B; n > 1;) {
    const int half = n >> 1;
    if (__ldg(cu_q + lo + half) <= row)
      lo += half, n -= half;
    else
      n = half;
  }
  return row < __ldg(cu_q + lo + 1) ? lo : -1;
}

// Where a token goes (written by one warp, read by the block).
struct Place {
  int64_t page;   // its page (< 0: its K and V are dropped)
  int64_t table;  // row of cos and sin; < 0: no such row
  int at;         // row in the page
  int live;       // a row of some sequence
};

// INTER: pairs (2j, 2j + 1) instead of (j, j + rot / 2).
template <int D, PageFormat PAGES, bool INTER>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(PAGES)) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int H = D / 16;  // values of a chunk
  constexpr uint32_t kRowBytes = D * 2;
  constexpr bool FP8 = PAGES == kPagesFp8, FP4 = PAGES == kPagesFp4;
  constexpr bool kHoldTurns = PAGES == kPagesBf16;
  static_assert(!FP4 || H == 8, "a block is two chunks");
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t(*ring)[kGroups * kRowBytes] = reinterpret_cast<uint8_t(*)[kGroups * kRowBytes]>(smem);
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ Place places[kMaxTokens];
  // of each token of the run: its rows of cos, sin and -sin, then (fp8) the scales of its block
  float* turns = reinterpret_cast<float*>(smem + kStages * kGroups * kRowBytes);
  float* scales = turns + a.run_tokens * 3 * (a.rot >> 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = threadIdx.x & 7;
  const int n_heads = a.Hq + 2 * a.Hkv;  // queries, keys, values
  // this CTA's run of (token, head) pairs
  const uint32_t n_pairs = static_cast<uint32_t>(a.T) * n_heads;
  const uint32_t pair0 = blockIdx.x * static_cast<uint32_t>(a.steps * kGroups);
  const uint32_t pair1 = min(pair0 + static_cast<uint32_t>(a.steps * kGroups), n_pairs);
  const int steps = static_cast<int>((pair1 - pair0 + kGroups - 1) / kGroups);
  const int t0 = static_cast<int>(pair0 / n_heads);  // first token of the run
  const int tokens = static_cast<int>((pair1 - 1) / n_heads) - t0 + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kGroups);
    }
    fence_mbar_init();
  }
  __syncthreads();

  // (token, head) of this lane's (producer) or group's (consumer) pair; a stage on: kGroups pairs
  int t = 0, h = static_cast<int>(pair0 - static_cast<uint32_t>(t0) * n_heads) + (warp == kWarps ? lane : threadIdx.x >> 3);
  while (h >= n_heads) h -= n_heads, ++t;
  auto advance = [&]() {
    h += kGroups;
    while (h >= n_heads) h -= n_heads, ++t;
  };

  if (warp == kWarps) {
    // ------------------------------------------------------------ the copies
    int done = 0;
    for (int n = 0; n < steps; ++n, advance()) {
      const int s = n % kStages;
      const int valid = static_cast<int>(min(pair1 - pair0 - static_cast<uint32_t>(n * kGroups), static_cast<uint32_t>(kGroups)));
      if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((n / kStages) - 1) & 1, a.err, kDevErrEmptyWait))) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(valid) * kRowBytes);
      __syncwarp();
      // a copy for each head; heads of one projection in a row go in one
      const bool starts = a.fused ? lane == 0 || h == 0 : true;
      if (lane < valid && starts) {
        const int64_t row = t0 + t;
        const __nv_bfloat16* from = h < a.Hq           ? a.q + row * a.q_st + h * a.q_sh
                                    : h < a.Hq + a.Hkv ? a.k + row * a.k_st + (h - a.Hq) * a.k_sh
                                                       : a.v + row * a.v_st + (h - a.Hq - a.Hkv) * a.v_sh;
        const int heads = a.fused ? min(valid - lane, n_heads - h) : 1;
        bulk_load(&ring[s][lane * kRowBytes], from, heads * kRowBytes, &full[s]);
      }
      done = n + 1;
    }
    // every copy lands before the CTA may exit
    for (int n = max(0, done - kStages); n < done; ++n)
      if (!mbar_wait(&full[n % kStages], (n / kStages) & 1, a.err, kDevErrDrainWait)) break;
    return;
  }

  // this lane's two chunks.  Halves: values f.. and their partners; behind the rotated dims the
  // rest is split in two the same way.  Interleaved: pairs lie inside a chunk
  const int half = a.rot >> 1, f = l8 * H;
  const bool in_rot = f < half;
  const int c0 = INTER || in_rot ? f : a.rot + f - half;
  const int c1 = INTER ? D / 2 + f : in_rot ? f + half : a.rot + (D - a.rot) / 2 + f - half;
  const bool turn0 = INTER ? c0 < a.rot : in_rot, turn1 = INTER ? c1 < a.rot : in_rot;

  // fp4: where the other half of each chunk's block is
  ChunkAt mate0 = {0, 0}, mate1 = {0, 0};
  if constexpr (FP4) {
    mate0 = chunk_at<H>((c0 / H) ^ 1, INTER, a.rot);
    mate1 = chunk_at<H>((c1 / H) ^ 1, INTER, a.rot);
  }

  // Places: a lane for each token, so that the chains of loads of all tokens run side by side
  {
    const int i = warp + kWarps * lane, row = t0 + i;
    const bool mine = lane < kMaxTokens / kWarps && i < tokens;
    Place pl;
    pl.page = pl.table = -1;
    pl.at = 0;
    const int b = mine ? sequence_of(a.cu_q, a.B, row) : -1;
    pl.live = b >= 0;
    if (b >= 0) {
      // place in the sequence
      const int64_t pos = static_cast<int64_t>(max(__ldg(a.seq_lens + b), 0)) - min(__ldg(a.cu_q + b + 1), a.T) + row;
      pl.table = a.positions ? __ldg(a.positions + row) : pos;
      if (pos >= 0 && pos < static_cast<int64_t>(a.max_blocks) * a.block_len) {
        const int block = static_cast<int>(pos) / a.block_len;  // the capacity is below 2^31
        pl.page = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_blocks + block);
        pl.at = static_cast<int>(pos) - block * a.block_len;
        if (pl.page >= a.num_blocks) pl.page = -1;
      }
      if (pl.table >= a.max_pos) pl.table = -1;
      if (a.rot > 0 && pl.table < 0) atomicOr(a.err + kErrCode, static_cast<unsigned int>(kDevErrPosition));
    }
    if (mine) places[i] = pl;
    // lanes 0 .. 15: the row of cos, 16 .. 31: of sin
    const int n_mine = (tokens - warp + kWarps - 1) / kWarps, per = half >> 2, c4 = lane & 15;
    const float* table = lane < 16 ? a.cos : a.sin;
    const float nan = __int_as_float(0x7fc00000);
#pragma unroll 4
    for (int x = 0; x < n_mine; ++x) {
      const int64_t at = __shfl_sync(0xffffffffu, pl.table, x);
      const bool live = __shfl_sync(0xffffffffu, pl.live, x) != 0;
      if (live && c4 < per) {
        float4 u = make_float4(nan, nan, nan, nan);
        if (at >= 0) u = __ldg(reinterpret_cast<const float4*>(table + at * half) + c4);
        float4* to = reinterpret_cast<float4*>(turns + (warp + kWarps * x) * 3 * half) + c4;
        to[(lane >> 4) * per] = u;
        if (lane >= 16) to[2 * per] = make_float4(-u.x, -u.y, -u.z, -u.w);
      }
      if constexpr (FP8) {
        const int64_t page = __shfl_sync(0xffffffffu, pl.page, x);
        const int block = __shfl_sync(0xffffffffu, pl.at, x) / a.scale_block;
        if (page >= 0 && a.Hkv <= kScaleHeads && c4 < a.Hkv)
          scales[(warp + kWarps * x) * 2 * kScaleHeads + lane] =
              __ldg((lane < 16 ? a.k_scale : a.v_scale) + (page * a.Hkv + c4) * (a.block_len / a.scale_block) + block);
      }
    }
  }
  named_barrier(1, kWarps * 32);  // (the copying warp goes its own way)

  Place pl;
  pl.live = 0;
  int have_t = -1, have_w = -1;  // token of the place, kind of the weights held
  // halves: cs, sn, -sn of the chunk's values; interleaved: (c, c) and (-s, s) of its pairs
  uint64_t held_c[H], held_s[H], wt[H];
#pragma unroll
  for (int j = 0; j < H; ++j) held_c[j] = held_s[j] = wt[j] = 0ull;
  auto load_turns = [&](uint64_t(&cs)[H], uint64_t(&sn)[H]) {
    const float* c = turns + t * 3 * half;  // cos, sin, -sin
    if constexpr (INTER) {
#pragma unroll
      for (int j = 0; j < H; ++j)
        if (j < H / 2 ? turn0 : turn1) {
          const float* at = c + (j < H / 2 ? c0 + 2 * j : c1 + 2 * (j - H / 2)) / 2;
          cs[j] = pack2(at[0], at[0]);
          sn[j] = pack2(at[2 * half], at[half]);
        }
    } else if (turn0) {
#pragma unroll
      for (int j = 0; j < H / 2; j += 2) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(c + f + 2 * j);
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(c + half + f + 2 * j);
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(c + 2 * half + f + 2 * j);
        cs[j] = u.x, cs[j + 1] = u.y;
        sn[j] = v.x, sn[j + 1] = v.y;
        sn[H / 2 + j] = w.x, sn[H / 2 + j + 1] = w.y;
      }
    }
  };
  for (int n = 0; n < steps; ++n, advance()) {
    const int s = n % kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (n / kStages) & 1, a.err, kDevErrFullWait))) break;
    uint32_t r[H];
    {
      const uint8_t* row = &ring[s][(threadIdx.x >> 3) * kRowBytes];
      load_chunk<H>(reinterpret_cast<const __nv_bfloat16*>(row) + c0, r);
      load_chunk<H>(reinterpret_cast<const __nv_bfloat16*>(row) + c1, r + H / 2);
    }
    const bool here = pair0 + static_cast<uint32_t>(n * kGroups + (threadIdx.x >> 3)) < pair1;
    if (here && t != have_t) {  // a new token
      have_t = t;
      pl = places[t];
      if constexpr (kHoldTurns)
        if (pl.live) load_turns(held_c, held_s);
    }
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
    uint64_t x[H];  // chunk 0, chunk 1
#pragma unroll
    for (int j = 0; j < H; ++j) x[j] = pack2(bf16_lo(r[j]), bf16_hi(r[j]));
    // the sum of squares over the 8 lanes: whole warps, values included (unused there)
    uint64_t acc = 0ull;
#pragma unroll
    for (int j = 0; j < H; ++j) acc = fma2(x[j], x[j], acc);
    float ss = sum_f32x2(acc);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // the head is read: the sum that says so holds all its values
    if (l8 == 0) arrive_after(&empty[s], ss);
    // (shuffles below stay within the 8 lanes of a head, which leave here together or not at all)
    if (!here || !pl.live) continue;
    if (!is_v) {
      const void* wp = is_q ? a.q_weight : a.k_weight;
      const int64_t w_sh = is_q ? a.q_weight_sh : a.k_weight_sh;
      float inv = 1.f;
      if (wp) {
        if (w_sh != 0 || have_w != (is_q ? 0 : 1)) {
          const int64_t at = (is_q ? h : h - a.Hq) * w_sh;
          load_weight<H>(wp, a.weight_bf16 != 0, at + c0, wt);
          load_weight<H>(wp, a.weight_bf16 != 0, at + c1, wt + H / 2);
          have_w = is_q ? 0 : 1;
        }
        inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < H; ++j) x[j] = mul2(x[j], wt[j]);
      }
      auto rotate = [&](const uint64_t(&cs)[H], const uint64_t(&sn)[H]) {
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < H; ++j)
            if (j < H / 2 ? turn0 : turn1) x[j] = fma2(x[j], cs[j], mul2(swap2(x[j]), sn[j]));
        } else if (turn0) {
#pragma unroll
          for (int j = 0; j < H / 2; ++j) {
            const uint64_t u = x[j], v = x[H / 2 + j];
            x[j] = fma2(u, cs[j], mul2(v, sn[H / 2 + j]));
            x[H / 2 + j] = fma2(v, cs[j], mul2(u, sn[j]));
          }
        }
      };
      if constexpr (kHoldTurns) {
        rotate(held_c, held_s);
      } else {
        uint64_t cs[H], sn[H];
        load_turns(cs, sn);
        rotate(cs, sn);
      }
      const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
      for (int j = 0; j < H; ++j) x[j] = mul2(x[j], inv2);
      if (is_q || PAGES == kPagesBf16) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
          float u, v;
          unpack2(x[j], u, v);
          r[j] = pack_bf16(u, v);
        }
      }
    }
    if (is_q) {
      __nv_bfloat16* o = a.q_out + (t0 + static_cast<int64_t>(t)) * a.o_st + h * a.o_sh;
      store_chunk<H>(o + c0, r);
      store_chunk<H>(o + c1, r + H / 2);
    } else if (pl.page >= 0) {
      const int g = h - a.Hq - (is_v ? a.Hkv : 0);
      const int64_t to =
          pl.page * (is_v ? a.vp_sb : a.kp_sb) + g * (is_v ? a.vp_sh : a.kp_sh) + pl.at * (is_v ? a.vp_st : a.kp_st);
      if constexpr (FP8) {
        float scale;
        if (a.Hkv <= kScaleHeads)
          scale = scales[(2 * t + is_v) * kScaleHeads + g];
        else
          scale = __ldg((is_v ? a.v_scale : a.k_scale) + (pl.page * a.Hkv + g) * (a.block_len / a.scale_block) +
                        pl.at / a.scale_block);
        uint8_t* o = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + to;
        store_e4m3<H>(o + c0, x, scale);
        store_e4m3<H>(o + c1, x + H / 2, scale);
      } else if constexpr (FP4) {
        // magnitudes order as their bits, NaN above infinity
        uint32_t most0 = 0u, most1 = 0u;
#pragma unroll
        for (int j = 0; j < H / 2; ++j) {
          float u, v;
          unpack2(x[j], u, v);
          most0 = max(most0, max(__float_as_uint(u) & 0x7FFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu));
          unpack2(x[H / 2 + j], u, v);
          most1 = max(most1, max(__float_as_uint(u) & 0x7FFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu));
        }
        const unsigned eight = 0xFFu << (lane & 24);  // the head's lanes, which are all here
        const uint32_t u0 = __shfl_sync(eight, most0, mate0.lane, 8), u1 = __shfl_sync(eight, most1, mate0.lane, 8);
        const uint32_t v0 = __shfl_sync(eight, most0, mate1.lane, 8), v1 = __shfl_sync(eight, most1, mate1.lane, 8);
        most0 = max(most0, mate0.second ? u1 : u0);
        most1 = max(most1, mate1.second ? v1 : v0);
        uint8_t* o = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + to;
        uint8_t* sc = (is_v ? a.v_block : a.k_block) +
                      ((pl.page * a.Hkv + g) * a.block_len + pl.at) * static_cast<int64_t>(D / kFp4Block);
        const float hs = head_scale(is_v ? a.v_head : a.k_head, g);
        store_fp4(o + c0 / 2, (c0 & 8) ? nullptr : sc + c0 / kFp4Block, x, __uint_as_float(most0), hs);
        store_fp4(o + c1 / 2, (c1 & 8) ? nullptr : sc + c1 / kFp4Block, x + H / 2, __uint_as_float(most1), hs);
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(is_v ? a.v_pages : a.k_pages) + to;
        store_chunk<H>(o + c0, r);
        store_chunk<H>(o + c1, r + H / 2);
      }
    }
  }
}

template <int D, PageFormat PAGES>
cudaError_t launch(AppendArgs a, int sms, cudaStream_t stream) {
  const int64_t n_heads = a.Hq + 2 * a.Hkv, pairs = a.T * n_heads;
  // equal runs for the CTAs that are resident at once, of one stage at least; a run touches kMaxTokens tokens at most
  const int64_t runs = static_cast<int64_t>(sms) * ctas_per_sm(PAGES);
  int64_t steps = (pairs + kGroups * runs - 1) / (kGroups * runs);
  steps = std::min<int64_t>(steps, std::max<int64_t>(1, (kMaxTokens - 2) * n_heads / kGroups));
  a.steps = static_cast<int>(steps);
  a.fused = a.q_sh == D && a.k_st == a.q_st && a.v_st == a.q_st && a.k_sh == D && a.v_sh == D && a.k == a.q + a.Hq * D &&
            a.v == a.k + a.Hkv * D;
  const unsigned int blocks = static_cast<unsigned int>((pairs + steps * kGroups - 1) / (steps * kGroups));
  a.run_tokens = static_cast<int>((steps * kGroups + n_heads - 2) / n_heads + 1);
  const auto bytes = [](int tokens, int rot) {
    return kStages * kGroups * D * 2 + tokens * (rot / 2 * 3 + (PAGES == kPagesFp8 ? 2 * kScaleHeads : 0)) * 4;
  };
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [&] {
    cudaError_t x = cudaFuncSetAttribute(append_kernel<D, PAGES, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes(kMaxTokens, D));
    if (x != cudaSuccess) return x;
    return cudaFuncSetAttribute(append_kernel<D, PAGES, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bytes(kMaxTokens, D));
  });
  if (e != cudaSuccess) return e;
  const size_t smem = bytes(a.run_tokens, a.rot);
  if (a.interleaved)
    append_kernel<D, PAGES, true><<<blocks, kThreads, smem, stream>>>(a);
  else
    append_kernel<D, PAGES, false><<<blocks, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int32_t d, PageFormat pages, int sms, cudaStream_t stream) {
  if (d == 64) return launch<64, kPagesBf16>(a, sms, stream);
  if (pages == kPagesFp4) return launch<128, kPagesFp4>(a, sms, stream);
  return pages == kPagesFp8 ? launch<128, kPagesFp8>(a, sms, stream) : launch<128, kPagesBf16>(a, sms, stream);
}

}  // namespace skv
