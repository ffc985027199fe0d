// Attention of up to 8 rows (new token, head of the group) of a KV head over 4-bit pages: a decode step
// of groups of 8 heads or fewer (attn_chunk_paged, both passes of attn_shared_prefix_paged).
//
// The mathematics and the equal runs of KV tiles are those of chunk_rows.cu.  What differs: 4-bit tiles take
// the instructions that widen them (1500 a warp and tile with 16 rows, where HBM brings a tile every 390 cycles
// an SM), in chains that the warps have to cover, so the rows lie on the 8 columns of the products, not on their 16 rows:
//   S^T = K Q^T (16 tokens x 8 rows a product) and O^T = V^T P^T (16 dims x 8 rows), half the products, scores and
//   sums of O of a tile of 16 rows, half of which would be padding;
//   S^T's fragments, packed in pairs and turned by movmatrix, are P^T's operand;
//   the weights' maxima, factors and sums stay in the lanes that hold their rows of O;
//   a warp needs 128 registers, so that 16 warps an SM (two CTAs of 7 and a producer) cover each other's
//   chains of conversions, and they join at the end of an item all at once, each thread summing 4 columns of a
//   row over the warps.
//
// Measured: decode of 64 sequences of 4096 to 16384 tokens, 64 / 8 heads, 166 us (0.62 of the measured copy
// rate; 203 on the kernel of 16 rows; 8 instructions for 8 codes of K, 13 for 8 of V, at 2.1 a cycle: issue slots
// and the fullest pipe are half busy, so what bounds it is the latency of the chains beside the instructions' number).  Before the
// scales' loads were held ahead of the arrival (160): 5 warps a CTA 171, 6 176, 4 with ten stages 163; rings of their
// own for K and V, with K's freed after the scores, 171.
#include <cuda_runtime.h>

#include "chunk_plan.cuh"
#include "skv_common.cuh"
#include "skv_internal.h"
#include "warp_wait.cuh"

namespace skv {

namespace {

constexpr int kRows = 8;
constexpr int D = 128;
constexpr int TN = kTileN;
constexpr int WN = 7;      // consumer warps
constexpr int NSTAGE = 8;  // tiles in the ring
constexpr int kThreads = (WN + 1) * 32;
constexpr int kCtas = 2;   // an SM
constexpr int kTile = TN * D / 2, kScales = TN * D / kFp4Block;
constexpr int kStage = 2 * (kTile + kScales);  // K, V, K's scales, V's
// Full barriers are per consumer warp, DW of them each: a warp's wait is then always for the phase after the
// one it saw last
constexpr int DW = (NSTAGE + WN - 1) / WN, NFULL = WN * DW;
constexpr int kRowFloats = D + 4;  // (rows 2 tq apart by 32 bytes of the banks: stores of O without conflicts)
constexpr int OFF_O = NSTAGE * kStage;                      // each warp's O
constexpr int OFF_ML = OFF_O + WN * kRows * kRowFloats * 4;  // (m, l) of each warp's rows
constexpr int OFF_INFO = OFF_ML + WN * kRows * 8;            // factor and weight of the prefix of each row
constexpr int OFF_BAR = OFF_INFO + kRows * 8;
constexpr int OFF_RUN = OFF_BAR + 256;                       // each consumer warp's run and piece
constexpr int kSmem = 1024 + OFF_RUN + WN * 192;
static_assert((NFULL + NSTAGE) * 8 <= 256, "barriers");
static_assert(kCtas * (kSmem + 1536) <= 227 * 1024, "CTAs an SM");
constexpr float kUp = 14.f;  // weights are 2^kUp at most (see chunk_rows.cu)

__device__ __forceinline__ int full_slot(int x) { return (x % WN) * DW + (x / WN) % DW; }
__device__ __forceinline__ uint32_t full_parity(int x) { return static_cast<uint32_t>((x / WN) / DW) & 1u; }
// Byte `byte` of token `tok`'s row of a tile: 64-byte rows under the 64-byte swizzle.
__device__ __forceinline__ uint32_t tile_off(uint32_t tok, uint32_t byte) {
  return tok * 64u + ((((byte >> 4) ^ ((tok >> 1) & 3u)) << 4) | (byte & 15u));
}
__device__ __forceinline__ uint32_t half_mask(bool lo, bool hi) {
  return (lo ? 0x0000FFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
// (x0, x1) * s and (x0, x1) + s, packed.
__device__ __forceinline__ void mul2(float& x0, float& x1, uint64_t s) {
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%0, %1};\n\tmul.rn.f32x2 a, a, %2;\n\tmov.b64 {%0, %1}, a;\n\t}" : "+f"(x0), "+f"(x1) : "l"(s));
}
__device__ __forceinline__ void add2(float& x0, float& x1, uint64_t s) {
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%0, %1};\n\tadd.rn.f32x2 a, a, %2;\n\tmov.b64 {%0, %1}, a;\n\t}" : "+f"(x0), "+f"(x1) : "l"(s));
}
__device__ __forceinline__ void consumers_sync() { named_barrier(1, WN * 32); }

template <bool SHARED>
__global__ void __launch_bounds__(kThreads, kCtas)
    chunk_rows4_kernel(const __grid_constant__ PartialParams p, const __grid_constant__ ChunkMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + NFULL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NFULL; ++s) mbar_init(&full[s], 1);
    for (int s = 0; s < NSTAGE; ++s) mbar_init(&empty[s], 1);
    fence_mbar_init();
  }
  // (the passes of a shared prefix: see chunk_rows.cu)
  auto first_pass_done = [&]() {
    if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (SHARED && p.ck.whole) first_pass_done();
  using Runs = ChunkRuns<SHARED>;
  Runs runs;  // (synchronises the block)
  if (!chunk_find_runs<kThreads, SHARED>(p.ck, gridDim.x, blockIdx.x, &runs)) {
    first_pass_done();
    return;
  }

  if (warp == WN) {
    // ------------------------------------------------------------ producer warp
    // Pages and rows of 32 tiles at a time, a lane each
    if (lane == 0) {
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
      tma_prefetch_desc(&maps.k_block);
      tma_prefetch_desc(&maps.v_block);
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
          pages = chunk_page_of<SHARED>(p, pc.b, t);
          rows = t % p.block_len;
        }
        const int n = min(32, pc.n_tiles - i0);
        for (int i = 0; i < n; ++i) {
          const int page = __shfl_sync(0xffffffffu, pages, i), row = __shfl_sync(0xffffffffu, rows, i);
          const int s = x % NSTAGE;
          if (lane == 0) {
            ok = x < NSTAGE || mbar_wait(&empty[s], ((x / NSTAGE) - 1) & 1, p.err, kDevErrEmptyWait);
            if (ok) {
              uint64_t* fb = &full[full_slot(x)];
              mbar_arrive_expect_tx(fb, kStage);
              uint8_t* ks = smem + s * kStage;
              tma_load_4d(ks, &maps.k, fb, 0, row, pc.g, page, pol);
              tma_load_4d(ks + kTile, &maps.v, fb, 0, row, pc.g, page, pol);
              tma_load_4d(ks + 2 * kTile, &maps.k_block, fb, row * (D / kFp4Block / 4), pc.g, page, 0, pol);
              tma_load_4d(ks + 2 * kTile + kScales, &maps.v_block, fb, row * (D / kFp4Block / 4), pc.g, page, 0, pol);
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
      if (!mbar_wait(&full[full_slot(y)], full_parity(y), p.err, kDevErrDrainWait)) break;
    first_pass_done();
    return;
  }

  // -------------------------------------------------------------- consumer warps
  const int gq = lane >> 2, tq = lane & 3, mi = lane >> 3;
  float2* ml = reinterpret_cast<float2*>(smem + OFF_ML);
  float2* info = reinterpret_cast<float2*>(smem + OFF_INFO);
  static_assert(sizeof(Runs) <= 64 && sizeof(ChunkPiece) <= 128, "a warp's place");
  Runs* run = reinterpret_cast<Runs*>(smem + OFF_RUN + warp * 192);
  ChunkPiece& pc = *reinterpret_cast<ChunkPiece*>(smem + OFF_RUN + warp * 192 + 64);
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
  // A warp that gave up a wait takes no further tile, but goes on through the pieces, since the others count
  // on it at their barriers
  WarpWait wait(p.err);
  while (next_piece()) {
    const int rows_total = pc.n * p.G, m0 = pc.mt * kRows;
    // ---- Q (B operand, 8 rows): row gq's dims 8 tq .. 8 tq + 7 of each chunk of 32, in fp16 times the power of two
    // that puts the row's largest magnitude in [2^14, 2^15); the power goes back into the score's scale
    uint32_t qb[D / 16][2];
    float q_scale;
    {
      const int m = m0 + gq;
      const bool valid = m < rows_total;
      const int t = valid ? m / p.G : 0, h = pc.g * p.G + (valid ? m % p.G : 0);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (pc.row0 + static_cast<int64_t>(t)) * p.q_st + h * p.q_sh + 8 * tq;
      uint4 u[D / 32];
      uint32_t most = 0u;  // magnitudes order as their bits
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        u[c] = valid ? *reinterpret_cast<const uint4*>(q + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (uint32_t w : {u[c].x, u[c].y, u[c].z, u[c].w}) most = max(most, max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
      }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const bool finite = most < 0x7F800000u;
      const int qe = most == 0u ? 0 : min(max(static_cast<int>(most >> 23) - 127 - 14, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - qe) << 23);
      q_scale = finite ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + qe) << 23) : __int_as_float(0x7fc00000);
      q_scale *= head_scale(p.k_head, pc.g);
      auto narrow = [&](uint32_t w) { return pack_f16(bf16_lo(w) * down, bf16_hi(w) * down); };
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        qb[2 * c][0] = narrow(u[c].x), qb[2 * c][1] = narrow(u[c].y);
        qb[2 * c + 1][0] = narrow(u[c].z), qb[2 * c + 1][1] = narrow(u[c].w);
      }
    }
    // this lane's rows of the scores and of O: 2 tq and 2 tq + 1
    const int pos0 = chunk_pos0<SHARED>(p.ck, pc.n, pc.m), pos_step = chunk_pos_step<SHARED>(p.ck);
    auto window_lo = [&](int pos) -> int { return p.ck.window > 0 && pos >= p.ck.window ? pos - p.ck.window + 1 : 0; };
    int hz[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) hz[r] = pos0 + min(m0 + 2 * tq + r, rows_total - 1) / p.G * pos_step;
    const int hz_min = pos0 + m0 / p.G * pos_step;
    const int wl_max = window_lo(pos0 + min(m0 + kRows - 1, rows_total - 1) / p.G * pos_step);
    const uint64_t sl = pack2(__shfl_sync(0xffffffffu, q_scale, 8 * tq), __shfl_sync(0xffffffffu, q_scale, 8 * tq + 4));

    float o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};

    // this warp's tiles: those whose number in the CTA is `warp` modulo WN
    for (int i = (warp + WN - x0 % WN) % WN; i < pc.n_tiles; i += WN) {
      const int x = x0 + i, s = x % NSTAGE;
      const int t0 = pc.token(i);
      if (!wait(&full[full_slot(x)], full_parity(x), kDevErrFullWait)) break;
      const uint32_t kbase = smem_u32(smem + s * kStage), vbase = kbase + kTile;

      // ---- S^T = K Q^T: of 16 tokens a lane has gq and gq + 8, of each chunk of 32 dims 8 tq .. 8 tq + 7, which lie
      // in one block.  Code times block scale is exact in fp16
      float st[TN / 16][4];
#pragma unroll
      for (int np = 0; np < TN / 16; ++np) st[np][0] = st[np][1] = st[np][2] = st[np][3] = 0.f;
      {
        const uint8_t* ksb = smem + s * kStage + 2 * kTile + gq * (D / kFp4Block);
#pragma unroll
        for (int np = 0; np < TN / 16; np += 2) {
#pragma unroll
          for (int c2 = 0; c2 < D / 64; ++c2) {
            uint32_t w[4][2], by[4];  // [8 tokens][chunk], the scales of the two chunks' blocks
#pragma unroll
            for (int h = 0; h < 4; h += 2)
              ldsm_x4(kbase + tile_off(16 * np + (h + (mi >> 1)) * 8 + (lane & 7), (2 * c2 + (mi & 1)) * 16), w[h][0], w[h][1],
                      w[h + 1][0], w[h + 1][1]);
#pragma unroll
            for (int h = 0; h < 4; ++h)
              by[h] = e4m3x2_low_to_f16x2(prmt(
                  ring_load(ksb + (16 * np + 8 * h) * (D / kFp4Block) + 4 * c2), 0u, (tq >> 1) ? 0x31u : 0x20u));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t k[4][4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const uint32_t b = prmt(by[h], 0u, c ? 0x3232u : 0x1010u);
                e2m1x8_to_f16x2x4(w[h][c], k[h][0], k[h][1], k[h][2], k[h][3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) k[h][j] = mul_f16x2(k[h][j], b);
              }
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 4; h += 2) {
                  const uint32_t a[4] = {k[h][2 * j], k[h + 1][2 * j], k[h][2 * j + 1], k[h + 1][2 * j + 1]};
                  const uint32_t* b = qb[4 * c2 + 2 * c + j];
                  mma_f16(st[np + (h >> 1)], a, b[0], b[1]);
                }
            }
          }
        }
      }

      // ---- scale, mask, online softmax
      const int r_lo = pc.tl.lo, r_hi = pc.tl.hi, sinks = pc.tl.sinks;
      const bool in_range = (t0 >= r_lo && t0 + TN <= r_hi) || t0 + TN <= sinks;
      const bool need_mask = !in_range || t0 + TN - 1 > hz_min || (t0 < wl_max && t0 + TN > sinks);
      auto in_item = [&](int tok) -> bool { return (tok >= r_lo && tok < r_hi) || tok < sinks; };
      float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int np = 0; np < TN / 16; ++np) {
        mul2(st[np][0], st[np][1], sl);
        mul2(st[np][2], st[np][3], sl);
      }
      if (need_mask) {
        const int wl[2] = {window_lo(hz[0]), window_lo(hz[1])};
#pragma unroll
        for (int np = 0; np < TN / 16; ++np)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = t0 + 16 * np + 8 * (e >> 1) + gq, r = e & 1;
            if (!(tok < r_hi && tok <= hz[r] && (tok >= wl[r] || tok < sinks))) st[np][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int np = 0; np < TN / 16; ++np)
#pragma unroll
        for (int r = 0; r < 2; ++r) tmax[r] = fmax3(tmax[r], st[np][r], st[np][2 + r]);
      float base[2], alpha[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], w));
        const float mnew = fmaxf(mrun[r], tmax[r]);
        base[r] = (mnew == -INFINITY) ? 0.f : mnew;
        alpha[r] = fast_exp2(mrun[r] - base[r]);  // 0 when mrun = -inf
        mrun[r] = mnew;
        lrun[r] *= alpha[r];
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {  // a row's maximum moved
        const uint64_t a2 = pack2(alpha[0], alpha[1]);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          mul2(o[j][0], o[j][1], a2);
          mul2(o[j][2], o[j][3], a2);
        }
      }
      // (two steps: a very large maximum less kUp would be rounded, and not alike in all warps)
      const uint64_t less = pack2(-base[0], -base[1]), up = pack2(kUp, kUp);
      uint64_t sum = 0ull;
      uint32_t pt[TN / 16][2];
#pragma unroll
      for (int np = 0; np < TN / 16; ++np)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          add2(st[np][2 * h], st[np][2 * h + 1], less);
          add2(st[np][2 * h], st[np][2 * h + 1], up);
          const float p0 = fast_exp2(st[np][2 * h]), p1 = fast_exp2(st[np][2 * h + 1]);
          sum = add_f32x2(sum, p0, p1);
          pt[np][h] = movmatrix_t(pack_f16(p0, p1));
        }
      {
        float s0, s1;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sum));
        lrun[0] += s0;
        lrun[1] += s1;
      }

      // ---- O^T += V^T P^T; V rows that no row sees may hold anything: masked in the tiles that have some
      auto pv = [&](auto vmasked) {
#pragma unroll
        for (int kk = 0; kk < TN / 16; ++kk) {
          uint32_t mlo = 0xFFFFFFFFu, mhi = 0xFFFFFFFFu;
          if constexpr (decltype(vmasked)::value) {
            const int ta = t0 + 16 * kk + 2 * tq, tb = ta + 8;
            mlo = half_mask(in_item(ta), in_item(ta + 1));
            mhi = half_mask(in_item(tb), in_item(tb + 1));
          }
          // ldmatrix.trans (16-bit view) gives a lane 4 dims of two tokens; of dims 32 c + 4 gq + i the nibbles of
          // both tokens make one byte, and so one pair.  Row gq of the product's tiles 2 c and 2 c + 1 is dim
          // 4 gq or 4 gq + 2, row gq + 8 the next one
          const uint8_t* vsb = smem + s * kStage + 2 * kTile + kScales + (16 * kk + 2 * tq) * (D / kFp4Block);
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
            const uint32_t moved = prmt(w >> 12, w << 12, 0x7610u);
            e2m1x8_to_f16x2x4((w & 0xF0F00F0Fu) | (moved & 0x0F0FF0F0u), f[0], f[2], f[1], f[3]);
          };
          uint32_t w[2][2];  // [chunk & 1][8 tokens]
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            if ((c & 1) == 0)
              ldsm_x4_t(vbase + tile_off(16 * kk + (mi & 1) * 8 + (lane & 7), (c + (mi >> 1)) * 16), w[0][0], w[0][1], w[1][0],
                        w[1][1]);
            uint32_t f[2][4];
            pairs(w[c & 1][0], f[0]);
            pairs(w[c & 1][1], f[1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[0][j] = mul_f16x2(f[0][j], sv[0][c]);
              f[1][j] = mul_f16x2(f[1][j], sv[1][c]);
              if constexpr (decltype(vmasked)::value) f[0][j] &= mlo, f[1][j] &= mhi;  // (the scales may be anything too)
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a[4] = {f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1]};
              mma_f16(o[2 * c + j], a, pt[kk][0], pt[kk][1]);
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

    // ---- join: (m, l) of every warp's rows, then O, every thread 4 columns of a row
    const bool direct = pc.slot < 0, behind = SHARED && direct && pc.skip > 0;
    auto out_row = [&](int r) -> int64_t {  // r < rows_total - m0
      const int m = m0 + r;
      return direct ? (pc.row0 + static_cast<int64_t>(m / p.G)) * p.Hq + pc.g * p.G + m % p.G
                    : static_cast<int64_t>(pc.slot) * kRows + r;
    };
    float4 before[2];  // of the prefix's rows, on their way under the join
    float before_lse[2] = {-INFINITY, -INFINITY};
    if constexpr (SHARED) {
      if (behind) {
        first_pass_done();
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int at = threadIdx.x + y * WN * 32;
          before[y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (at < kRows * D / 4 && m0 + (at >> 5) < rows_total)
            before[y] = __ldcg(reinterpret_cast<const float4*>(p.ck.prior_o + out_row(at >> 5) * D) + (at & 31));
          if (warp == 0 && m0 + 2 * tq + y < rows_total) before_lse[y] = __ldcg(p.ck.prior_lse + out_row(2 * tq + y));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) lrun[r] += __shfl_xor_sync(0xffffffffu, lrun[r], w);
      if (gq == 0) ml[warp * kRows + 2 * tq + r] = make_float2(mrun[r], lrun[r]);
    }
    consumers_sync();
    float M[2], L[2], f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      M[r] = -INFINITY;
#pragma unroll
      for (int w = 0; w < WN; ++w) M[r] = fmaxf(M[r], ml[w * kRows + 2 * tq + r].x);
      const float b = M[r] == -INFINITY ? 0.f : M[r];
      L[r] = 0.f;  // a NaN among the scores keeps it NaN, and the row is NaN
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float2 u = ml[w * kRows + 2 * tq + r];
        L[r] += u.y * fast_exp2(u.x - b);
      }
      f[r] = fast_exp2(mrun[r] - b);  // (a warp without a tile has O = 0; 0 * 2^-inf = 0)
    }
    float* obuf = reinterpret_cast<float*>(smem + OFF_O) + warp * kRows * kRowFloats;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float4*>(obuf + (2 * tq + r) * kRowFloats + 32 * c + 4 * gq) =
            make_float4(o[2 * c][r] * f[r], o[2 * c][2 + r] * f[r], o[2 * c + 1][r] * f[r], o[2 * c + 1][2 + r] * f[r]);
    if (warp == 0 && gq == 0) {
      constexpr float kLn2 = 0.6931471805599453f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool some = L[r] != 0.f;
        float lse = some ? (M[r] + (__log2f(L[r]) - kUp)) * kLn2 : -INFINITY;
        float inv = some ? head_scale(p.v_head, pc.g) / L[r] : 0.f, weight = 0.f;
        if (behind) {
          const ChunkJoin j = chunk_join(lse, before_lse[r]);
          inv *= j.own, weight = j.prior, lse = j.lse;
        }
        info[2 * tq + r] = make_float2(inv, weight);
        if (m0 + 2 * tq + r < rows_total) (direct ? p.ck.lse : p.out_lse)[out_row(2 * tq + r)] = lse;
      }
    }
    consumers_sync();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int at = threadIdx.x + y * WN * 32, row = at >> 5, c4 = at & 31;
      if (at >= kRows * D / 4 || m0 + row >= rows_total) continue;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(smem + OFF_O + (w * kRows + row) * kRowFloats * 4 + 16 * c4);
        u.x += z.x, u.y += z.y, u.z += z.z, u.w += z.w;
      }
      const float2 by = info[row];
      u.x *= by.x, u.y *= by.x, u.z *= by.x, u.w *= by.x;
      if (behind) {
        u.x = fmaf(before[y].x, by.y, u.x), u.y = fmaf(before[y].y, by.y, u.y);
        u.z = fmaf(before[y].z, by.y, u.z), u.w = fmaf(before[y].w, by.y, u.w);
      }
      const int64_t to = out_row(row) * D + 4 * c4;
      if (!direct)
        *reinterpret_cast<float4*>(p.out_o + to) = u;
      else if (SHARED && p.ck.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.ck.out) + to) = u;
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.ck.out) + to) = make_uint2(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w));
    }
    // (the next piece writes ml ahead of its first sync, whose readers here are behind the second; O and info after it)
  }
  first_pass_done();
}

template <bool SHARED>
cudaError_t launch(const PartialParams& p, const ChunkMaps& maps, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};  // per device
  cudaError_t e0 = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(chunk_rows4_kernel<SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e0 != cudaSuccess) return e0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(p.ck.n_wave));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (SHARED) {  // a programmatic dependent of the kernel before
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, chunk_rows4_kernel<SHARED>, p, maps);
}

}  // namespace

int chunk_rows4_rows() { return kRows; }
int chunk_rows4_ctas_per_sm() { return kCtas; }

cudaError_t launch_chunk_rows4(const PartialParams& p, const ChunkMaps& maps, cudaStream_t stream) {
  return p.ck.shared ? launch<true>(p, maps, stream) : launch<false>(p, maps, stream);
}

}  // namespace skv
