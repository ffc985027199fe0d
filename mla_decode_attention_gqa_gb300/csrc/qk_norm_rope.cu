// Norm of every query and key head, position rotation, and the write into the paged cache, in
// one pass over the new tokens (qk_norm_rope_append).
//
// For each token and head x in R^d:   y = x w / sqrt(mean(x^2) + eps)   (queries and keys),
//   (y_a, y_b) <- (y_a cos_j - y_b sin_j, y_b cos_j + y_a sin_j)   for j < rot / 2, with
//   (a, b) = (j, j + rot/2), or (2j, 2j + 1) interleaved; cos_j, sin_j: the row of the token's
//   position in the caller's tables.  The query goes out in bf16, the key to its page row in
//   bf16 or as the e4m3 code of y / scale (the block scale that the cache holds), the value
//   likewise without norm and rotation.  Everything between the loads and the one rounding at
//   the store is in fp32.
//
// Bound by HBM: each input is read once and each output written once.  16 lanes hold one head
// (d / 16 values each: 16 or 8 bytes a load), so the mean of squares is four shuffles and the
// rotation's partner value one shuffle; a 16-lane group keeps its token's cosines and sines in
// registers over kHeads heads, whose loads are all issued before the first is used.
#include <cuda_runtime.h>

#include "skv_common.cuh"
#include "skv_internal.h"

namespace skv {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // 16-lane groups of a block

// This lane's E values of a head row as floats.
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, uint32_t (&w)[E / 2]) {
  if constexpr (E == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}

template <int E>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&x)[E]) {
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// e4m3 codes of x / scale, saturated at +-448; a scale that is not a positive number stores
// zeros (the value that such a block stands for).
template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[E], float scale) {
  uint32_t w[E / 4];
  const bool ok = scale > 0.f && scale <= 3.402823466e38f;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 v = ok ? make_float2(__fdiv_rn(x[4 * i + 2 * j], scale), __fdiv_rn(x[4 * i + 2 * j + 1], scale))
                          : make_float2(0.f, 0.f);
      codes |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)) << (16 * j);
    }
    w[i] = codes;
  }
  if constexpr (E == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

template <int E, bool BF16>
__device__ __forceinline__ void load_weight(const void* w, int64_t at, float (&x)[E]) {
  if constexpr (BF16) {
    uint32_t u[E / 2];
    load_row<E>(static_cast<const __nv_bfloat16*>(w) + at, u);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[2 * i] = bf16_lo(u[i]), x[2 * i + 1] = bf16_hi(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at + i);
      x[i] = u.x, x[i + 1] = u.y, x[i + 2] = u.z, x[i + 3] = u.w;
    }
  }
}

// Sequence of packed row `row`: the b with cu_q[b] <= row < cu_q[b + 1], or -1.
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int row) {
  int lo = 0, hi = B;  // the number of sequences whose rows begin at or before `row`
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu_q + mid) <= row) lo = mid + 1; else hi = mid;
  }
  return (lo > 0 && row < __ldg(cu_q + lo)) ? lo - 1 : -1;
}

// FP8: e4m3 pages; HEADS: heads that one 16-lane group works off.
template <int D, bool FP8, int HEADS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int E = D / 16;
  const int l16 = threadIdx.x & 15;
  const int n_heads = a.Hq + 2 * a.Hkv;  // queries, keys, values
  const int parts = (n_heads + HEADS - 1) / HEADS;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x >> 4);
  const int64_t n_units = static_cast<int64_t>(a.T) * parts;
  // every lane stays to the end: the shuffles below take whole warps
  const bool live = unit < n_units;
  const int row = live ? static_cast<int>(unit / parts) : 0;
  const int h0 = live ? static_cast<int>(unit % parts) * HEADS : n_heads;

  // all loads of the group's heads first
  uint32_t raw[HEADS][E / 2];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    const __nv_bfloat16* p = nullptr;
    if (h < a.Hq)
      p = a.q + row * a.q_st + h * a.q_sh;
    else if (h < a.Hq + a.Hkv)
      p = a.k + row * a.k_st + (h - a.Hq) * a.k_sh;
    else if (h < n_heads)
      p = a.v + row * a.v_st + (h - a.Hq - a.Hkv) * a.v_sh;
    if (p) {
      load_row<E>(p + l16 * E, raw[i]);
    } else {
#pragma unroll
      for (int j = 0; j < E / 2; ++j) raw[i][j] = 0u;
    }
  }

  const int b = live ? sequence_of(a.cu_q, a.B, row) : -1;
  int64_t pos = -1;  // logical position in the sequence
  if (b >= 0) pos = static_cast<int64_t>(__ldg(a.seq_lens + b)) - __ldg(a.cu_q + b + 1) + row;
  // page row of the new token (page < 0: its K and V are dropped)
  int64_t page = -1;
  int at = 0;
  if (b >= 0 && h0 + HEADS > a.Hq && pos >= 0 && pos < static_cast<int64_t>(a.max_blocks) * a.block_len) {
    page = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_blocks + pos / a.block_len);
    at = static_cast<int>(pos % a.block_len);
    if (page >= a.num_blocks) page = -1;
  }
  // the rotation of this lane's values
  float cs[E], sn[E];
  const int d0 = l16 * E, half = a.rot >> 1;
  const bool turns = d0 < a.rot;  // rot is a multiple of 2 E: a lane turns all its values or none
  // interleaved pairs lie inside the lane; halves lie half / E lanes apart
  const bool upper = d0 >= half;
  const int partner = a.interleaved || !turns ? l16 : l16 + (upper ? -half / E : half / E);
#pragma unroll
  for (int j = 0; j < E; ++j) cs[j] = 1.f, sn[j] = 0.f;
  if (turns && b >= 0 && h0 < a.Hq + a.Hkv) {
    const int64_t rp = a.positions ? __ldg(a.positions + row) : pos;
    if (rp >= 0 && rp < a.max_pos) {
      const float* c = a.cos + rp * half;
      const float* s = a.sin + rp * half;
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          cs[j] = __ldg(c + d0 / 2 + j / 2);
          sn[j] = __ldg(s + d0 / 2 + j / 2);
        }
      } else {
        const int j0 = upper ? d0 - half : d0;
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(c + j0 + j));
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(s + j0 + j));
          cs[j] = c4.x, cs[j + 1] = c4.y, cs[j + 2] = c4.z, cs[j + 3] = c4.w;
          sn[j] = s4.x, sn[j + 1] = s4.y, sn[j + 2] = s4.z, sn[j + 3] = s4.w;
        }
      }
    } else {  // no such row of the tables: NaN, and the host is told
#pragma unroll
      for (int j = 0; j < E; ++j) cs[j] = sn[j] = __int_as_float(0x7fc00000);
      if (l16 == 0) atomicOr(a.err + kErrCode, static_cast<unsigned int>(kDevErrPosition));
    }
  }
  const int64_t weight_at = d0;

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
    float x[E];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) x[2 * j] = bf16_lo(raw[i][j]), x[2 * j + 1] = bf16_hi(raw[i][j]);
    // the 16-lane sum of squares and the partner's values: whole warps, values included (their
    // results are not used), so that no lane of a warp is missing
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const void* wp = is_q ? a.q_weight : a.k_weight;
    if (!is_v && wp) {
      const float inv = rsqrtf(ss * (1.f / D) + a.eps);
      float w[E];
      const int64_t wa = weight_at + (is_q ? h * a.q_weight_sh : (h - a.Hq) * a.k_weight_sh);
      if (a.weight_bf16)
        load_weight<E, true>(wp, wa, w);
      else
        load_weight<E, false>(wp, wa, w);
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = x[j] * inv * w[j];
    }
    float y[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float other = __shfl_sync(0xffffffffu, x[j], partner, 16);
      if (!turns || is_v) {
        y[j] = x[j];
      } else if (a.interleaved) {
        y[j] = (j & 1) ? fmaf(x[j], cs[j], x[j ^ 1] * sn[j]) : fmaf(x[j], cs[j], -x[j ^ 1] * sn[j]);
      } else {
        y[j] = upper ? fmaf(x[j], cs[j], other * sn[j]) : fmaf(x[j], cs[j], -other * sn[j]);
      }
    }
    if (b < 0 || h >= n_heads) continue;  // (no shuffle below)
    if (is_q) {
      store_bf16<E>(a.q_out + row * a.o_st + h * a.o_sh + d0, y);
    } else if (page >= 0) {
      const int g = h - a.Hq - (is_v ? a.Hkv : 0);
      const int64_t to = page * (is_v ? a.vp_sb : a.kp_sb) + g * (is_v ? a.vp_sh : a.kp_sh) +
                         at * (is_v ? a.vp_st : a.kp_st) + d0;
      if constexpr (FP8) {
        const int per = a.block_len / a.scale_block;
        const float sc = __ldg((is_v ? a.v_scale : a.k_scale) + (page * a.Hkv + g) * per + at / a.scale_block);
        store_e4m3<E>(static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + to, y, sc);
      } else {
        store_bf16<E>(static_cast<__nv_bfloat16*>(is_v ? a.v_pages : a.k_pages) + to, y);
      }
    }
  }
}

template <int D, bool FP8, int HEADS>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  const int64_t parts = (a.Hq + 2 * a.Hkv + HEADS - 1) / HEADS;
  const int64_t blocks = (a.T * parts + kGroups - 1) / kGroups;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  append_kernel<D, FP8, HEADS><<<static_cast<unsigned int>(blocks), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int32_t d, bool fp8, cudaStream_t stream) {
  if (d == 64) return launch<64, false, 4>(a, stream);
  return fp8 ? launch<128, true, 4>(a, stream) : launch<128, false, 4>(a, stream);
}

}  // namespace skv
