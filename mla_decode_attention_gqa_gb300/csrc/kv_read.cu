// Tokens of a paged cache as packed bf16 rows (kv_read_paged): what goes round a ring, or into a
// cache of another format.
//
// Packed row cu[b] + i is token starts[b] + i of sequence b; of every KV head its K and V rows:
// bf16 as they are; e4m3 code * block scale; e2m1 code * e4m3 block scale (exact) * head scale, in
// fp32, rounded once.
//
// Bound by HBM: pages in once, rows out once.  A lane takes 16 dims of a row (a 4-bit block: 8 bytes
// of codes, a scale, 32 bytes out), so that 8 lanes (heads of 64: 4) read a row and a warp reads the
// rows of neighbouring tokens, which lie side by side in the page, and writes whole rows.  Each
// lane has kAhead rows of its token on their way, K and V of some heads; the places of a
// block's tokens are found once, a lane each.  Measured: 8 histories of 20000 to 65536 4-bit tokens, 8 heads, 342 us
// (5.8 TB/s, 0.85 of the measured copy rate); blocks of 128 threads 350, of 256 369, of 512 432; 8 rows ahead 430.
#include <cuda_runtime.h>

#include <algorithm>

#include "skv_common.cuh"
#include "skv_internal.h"

namespace skv {

namespace {

constexpr int kThreads = 64;
constexpr int kAhead = 4;  // rows that a lane loads before it stores the first

// Where a packed row comes from.
struct Source {
  int64_t page;  // < 0: zeros
  int at;        // row in the page
  int live;      // a row of some sequence
};

template <PageFormat PAGES>
struct Loaded {
  uint4 u, v;  // bf16: 16 values; fp8: 16 codes (u); fp4: 16 codes (u.x, u.y)
  float scale;
};

template <int D, PageFormat PAGES>
__device__ __forceinline__ Loaded<PAGES> load_row(const ReadArgs& a, const Source& s, int g, bool is_v, int dim) {
  Loaded<PAGES> r;
  r.u = r.v = make_uint4(0u, 0u, 0u, 0u);
  r.scale = 0.f;
  if (s.page < 0) return r;
  const int64_t row = s.page * (is_v ? a.vp_sb : a.kp_sb) + g * (is_v ? a.vp_sh : a.kp_sh) + s.at * (is_v ? a.vp_st : a.kp_st);
  const uint8_t* pages = static_cast<const uint8_t*>(is_v ? a.v_pages : a.k_pages);
  if constexpr (PAGES == kPagesBf16) {
    const uint4* p = reinterpret_cast<const uint4*>(pages + 2 * (row + dim));
    r.u = __ldg(p);
    r.v = __ldg(p + 1);
  } else if constexpr (PAGES == kPagesFp8) {
    r.u = __ldg(reinterpret_cast<const uint4*>(pages + row + dim));
    r.scale = __ldg((is_v ? a.v_scale : a.k_scale) + (s.page * a.Hkv + g) * (a.block_len / a.scale_block) + s.at / a.scale_block);
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(pages + row + dim / 2));
    r.u.x = u.x, r.u.y = u.y;
    const uint32_t code = __ldg((is_v ? a.v_block : a.k_block) +
                                ((s.page * a.Hkv + g) * a.block_len + s.at) * static_cast<int64_t>(D / kFp4Block) + dim / kFp4Block);
    const uint32_t wide = e4m3x2_to_f16x2(static_cast<uint16_t>(code));
    r.scale = __low2float(*reinterpret_cast<const __half2*>(&wide));
  }
  return r;
}

__device__ __forceinline__ uint32_t scaled_pair(uint32_t f16x2, float block, float head) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
  return pack_bf16(f.x * block * head, f.y * block * head);
}

template <PageFormat PAGES>
__device__ __forceinline__ void store_row(const Loaded<PAGES>& r, float head, __nv_bfloat16* to) {
  uint32_t w[8];
  if constexpr (PAGES == kPagesBf16) {
    w[0] = r.u.x, w[1] = r.u.y, w[2] = r.u.z, w[3] = r.u.w;
    w[4] = r.v.x, w[5] = r.v.y, w[6] = r.v.z, w[7] = r.v.w;
  } else if constexpr (PAGES == kPagesFp8) {
    const uint32_t c[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2x2(c[i], lo, hi);
      w[2 * i] = scaled_pair(lo, r.scale, 1.f);
      w[2 * i + 1] = scaled_pair(hi, r.scale, 1.f);
    }
  } else {
    e2m1x8_to_f16x2x4(r.u.x, w[0], w[1], w[2], w[3]);
    e2m1x8_to_f16x2x4(r.u.y, w[4], w[5], w[6], w[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = scaled_pair(w[i], r.scale, head);
  }
  uint4* p = reinterpret_cast<uint4*>(to);
  __stcs(p, make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(p + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// blockIdx.x: tokens; blockIdx.y: a share of the heads, K and V of each.
template <int D, PageFormat PAGES>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ ReadArgs a, int heads_each) {
  constexpr int kLanes = D / 16, kTokens = kThreads / kLanes;
  static_assert(kTokens <= kThreads, "a thread for each token's place");
  __shared__ Source sources[kTokens];
  const int t0 = blockIdx.x * kTokens;
  if (threadIdx.x < kTokens) {
    const int row = t0 + threadIdx.x;
    Source s;
    s.page = -1;
    s.at = 0;
    s.live = 0;
    if (row < a.T && __ldg(a.cu) <= row) {
      int lo = 0;  // the last b with cu[b] <= row
      for (int n = a.B; n > 1;) {
        const int half = n >> 1;
        if (__ldg(a.cu + lo + half) <= row)
          lo += half, n -= half;
        else
          n = half;
      }
      if (row < __ldg(a.cu + lo + 1)) {
        s.live = 1;
        const int64_t pos = static_cast<int64_t>(row) - __ldg(a.cu + lo) + (a.starts ? __ldg(a.starts + lo) : 0);
        if (pos >= 0 && pos < static_cast<int64_t>(a.max_blocks) * a.block_len) {
          const int block = static_cast<int>(pos) / a.block_len;  // the capacity is below 2^31
          const int64_t page = __ldg(a.block_table + static_cast<int64_t>(lo) * a.max_blocks + block);
          s.at = static_cast<int>(pos) - block * a.block_len;
          if (page >= 0 && page < a.num_blocks) s.page = page;
        }
      }
    }
    sources[threadIdx.x] = s;
  }
  __syncthreads();
  const int tok = threadIdx.x / kLanes, dim = (threadIdx.x % kLanes) * 16;
  const Source s = sources[tok];
  if (!s.live) return;
  const int64_t t = t0 + tok;
  const int x0 = 2 * blockIdx.y * heads_each, x1 = min(x0 + 2 * heads_each, 2 * a.Hkv);  // 2 g + (V?)
  for (int x = x0; x < x1; x += kAhead) {
    Loaded<PAGES> r[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (x + i < x1) r[i] = load_row<D, PAGES>(a, s, (x + i) >> 1, ((x + i) & 1) != 0, dim);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (x + i < x1) {
        const int g = (x + i) >> 1;
        const bool is_v = ((x + i) & 1) != 0;
        const float head = PAGES == kPagesFp4 ? head_scale(is_v ? a.v_head : a.k_head, g) : 1.f;
        store_row<PAGES>(r[i], head, (is_v ? a.v_out + t * a.vo_st + g * a.vo_sh : a.k_out + t * a.ko_st + g * a.ko_sh) + dim);
      }
  }
}

template <int D, PageFormat PAGES>
cudaError_t launch(const ReadArgs& a, int sms, cudaStream_t stream) {
  constexpr int kTokens = kThreads / (D / 16);
  const int64_t blocks = (static_cast<int64_t>(a.T) + kTokens - 1) / kTokens;
  // few tokens: the heads are dealt to several blocks, down to kAhead rows of a lane each
  int parts = static_cast<int>(std::min<int64_t>((4 * sms + blocks - 1) / blocks, (2 * a.Hkv + kAhead - 1) / kAhead));
  const int heads_each = (a.Hkv + parts - 1) / parts;
  parts = (a.Hkv + heads_each - 1) / heads_each;
  kv_read_kernel<D, PAGES><<<dim3(static_cast<unsigned int>(blocks), parts), kThreads, 0, stream>>>(a, heads_each);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs& a, int32_t d, PageFormat pages, int sms, cudaStream_t stream) {
  if (d == 64) return launch<64, kPagesBf16>(a, sms, stream);
  if (pages == kPagesFp4) return launch<128, kPagesFp4>(a, sms, stream);
  return pages == kPagesFp8 ? launch<128, kPagesFp8>(a, sms, stream) : launch<128, kPagesBf16>(a, sms, stream);
}

}  // namespace skv
