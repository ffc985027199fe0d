// The plan and the merge of attention over ragged chunks (attn_chunk_paged).
//
// The merge joins partial rows: those of sequences whose KV tiles were dealt to several chunks
// (chunk_tc), or of items that a run's end cut (chunk_rows).
//
// For every such row, with k partials (o_c, lse_c): m = max lse_c, w_c = exp(lse_c - m),
// out = sum w_c o_c / sum w_c in bf16, lse = m + ln sum w_c; all partials empty: out = 0,
// lse = -inf.  Where they are stands in the plan (chunk_plan.cuh) of the call.  Of a shared prefix the
// result is fp32, and rows behind one are joined with it (ChunkArgs).
//
// Bound by the partials' bytes, which are mostly still in L2; what counts is how many loads
// are in flight.  A block takes 8 rows: one warp each while k <= 16 (all partials of a row in
// two batches of 8 loads), else one row after the other with the partials dealt to the 8
// warps, so that a single long sequence (hundreds of partials for a few rows) is not left to
// a few warps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "chunk_plan.cuh"
#include "skv_internal.h"

namespace skv {

namespace {

constexpr int kRowsPerBlock = 8;
constexpr int kWarpParts = 16;
constexpr int kBatch = 8;

// Running merge of one row's partials: this lane's 4 columns.
struct Joined {
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
};

// Partials first, first + step, .. below k of one row; at(c): the row of partial c.
template <int D, class At>
__device__ __forceinline__ Joined join(const float* part_o, const float* part_lse, At&& at, int first, int step, int k,
                                       int lane) {
  Joined j;
  bool nan = false;  // a NaN partial makes the row NaN (fmaxf drops it)
  for (int c = first + lane * step; c < k; c += 32 * step) {
    const float l = part_lse[at(c)];
    nan = nan || l != l;
    j.m = fmaxf(j.m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) j.m = fmaxf(j.m, __shfl_xor_sync(0xffffffffu, j.m, o));
  if (__any_sync(0xffffffffu, nan)) j.m = fmaxf(j.m, 0.f);
  if (j.m == -INFINITY) return j;
  for (int c0 = first; c0 < k; c0 += kBatch * step) {
    float w[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = c0 + u * step;
      const float l = c < k ? part_lse[at(c)] : -INFINITY;
      w[u] = l == -INFINITY ? 0.f : __expf(l - j.m);  // an empty partial's o was never written
      x[u] = (l != -INFINITY && 4 * lane < D) ? *reinterpret_cast<const float4*>(part_o + at(c) * D + 4 * lane)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      j.den += w[u];
      j.acc.x += w[u] * x[u].x;
      j.acc.y += w[u] * x[u].y;
      j.acc.z += w[u] * x[u].z;
      j.acc.w += w[u] * x[u].w;
    }
  }
  return j;
}

// (behind: the row's sequence has a prefix that another pass attended)
template <int D, bool SHARED>
__device__ __forceinline__ void store_row(const ChunkArgs& a, int64_t row, const Joined& j, int lane, bool behind) {
  float inv = j.den != 0.f ? 1.f / j.den : 0.f;
  float lse = j.den != 0.f ? j.m + logf(j.den) : -INFINITY;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (SHARED && behind) {
    const ChunkJoin both = chunk_join(lse, __ldcg(a.prior_lse + row));
    inv *= both.own;
    lse = both.lse;
    if (4 * lane < D) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.prior_o + row * D + 4 * lane));
      y = make_float4(x.x * both.prior, x.y * both.prior, x.z * both.prior, x.w * both.prior);
    }
  }
  if (4 * lane < D) {
    y = make_float4(fmaf(j.acc.x, inv, y.x), fmaf(j.acc.y, inv, y.y), fmaf(j.acc.z, inv, y.z), fmaf(j.acc.w, inv, y.w));
    if (SHARED && a.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + 4 * lane) = y;
    } else {
      __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y);
      __nv_bfloat162 hi = __floats2bfloat162_rn(y.z, y.w);
      uint2 u;
      u.x = *reinterpret_cast<uint32_t*>(&lo);
      u.y = *reinterpret_cast<uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + 4 * lane) = u;
    }
  }
  if (lane == 0) a.lse[row] = lse;
}

// One row's partials dealt to the block's warps.
template <int D>
struct BlockJoin {
  float m[kRowsPerBlock], den[kRowsPerBlock];
  float4 acc[kRowsPerBlock][D / 4];
};
template <int D, bool SHARED, class At>
__device__ __forceinline__ void join_by_block(const ChunkArgs& a, BlockJoin<D>& sm, const float* part_o,
                                              const float* part_lse, At&& at, int k, int64_t row, bool behind) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Joined j = join<D>(part_o, part_lse, at, warp, kRowsPerBlock, k, lane);
  __syncthreads();  // the sums before were read
  if (lane == 0) {
    sm.m[warp] = j.m;
    sm.den[warp] = j.den;
  }
  if (4 * lane < D) sm.acc[warp][lane] = j.acc;
  __syncthreads();
  if (warp == 0) {
    Joined s;
#pragma unroll
    for (int v = 0; v < kRowsPerBlock; ++v) s.m = fmaxf(s.m, sm.m[v]);
#pragma unroll
    for (int v = 0; v < kRowsPerBlock; ++v) {
      const float f = sm.m[v] == -INFINITY ? 0.f : __expf(sm.m[v] - s.m);
      s.den += f * sm.den[v];
      if (4 * lane < D) {
        const float4 x = sm.acc[v][lane];
        s.acc.x += f * x.x;
        s.acc.y += f * x.y;
        s.acc.z += f * x.z;
        s.acc.w += f * x.w;
      }
    }
    store_row<D, SHARED>(a, row, s, lane, behind);
  }
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
    chunk_merge_kernel(const __grid_constant__ ChunkArgs a, const float* part_o, const float* part_lse) {
  __shared__ int sm_parts[kRowsPerBlock], sm_n[kRowsPerBlock], sm_skip[kRowsPerBlock];
  __shared__ int64_t sm_row[kRowsPerBlock], sm_part[kRowsPerBlock];
  __shared__ BlockJoin<D> sm_join;
  // (the second pass of a shared prefix may start)
  if constexpr (SHARED) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the attention kernel before it on the stream is complete and its writes are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = a.Hkv * a.G;
  const int rows = __ldcg(a.plan + kPlanMerged);
  const int32_t* plan = a.plan + kPlanHead;
  for (int r0 = blockIdx.x * kRowsPerBlock; r0 < rows; r0 += gridDim.x * kRowsPerBlock) {
    const int r = r0 + warp;
    __syncthreads();  // the tables' earlier readers are done
    if (lane == 0) {
      int k = 0, n = 0, skip = 0;
      int64_t row = 0, part = 0;
      if (r < rows) {
        int lo = 0, hi = a.B - 1;  // the last sequence whose first row is <= r
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (__ldcg(plan + kPlanRow * mid + 1) <= r) lo = mid; else hi = mid - 1;
        }
        // sequences without rows to merge share the first row of the one after them
        const int in = r - __ldcg(plan + kPlanRow * lo + 1);
        int row0, m;
        chunk_lengths<SHARED>(a, lo, &row0, &n, &m, &skip);
        k = __ldcg(plan + kPlanRow * lo + 4);
        row = static_cast<int64_t>(row0) * Hq + in;
        part = static_cast<int64_t>(__ldcg(plan + kPlanRow * lo + 2)) + in;
      }
      sm_parts[warp] = k;
      sm_n[warp] = n;
      sm_skip[warp] = skip;
      sm_row[warp] = row;
      sm_part[warp] = part;
    }
    __syncthreads();
    int most = 0;
#pragma unroll
    for (int w = 0; w < kRowsPerBlock; ++w) most = max(most, sm_parts[w]);
    auto at = [&](int w) {
      const int64_t first = sm_part[w], stride = static_cast<int64_t>(sm_n[w]) * Hq;
      return [first, stride](int c) -> int64_t { return first + c * stride; };
    };
    if (most <= kWarpParts) {
      if (r < rows)
        store_row<D, SHARED>(a, sm_row[warp], join<D>(part_o, part_lse, at(warp), 0, 1, sm_parts[warp], lane), lane, sm_skip[warp] > 0);
    } else {
      for (int w = 0; w < kRowsPerBlock && r0 + w < rows; ++w)
        join_by_block<D, SHARED>(a, sm_join, part_o, part_lse, at(w), sm_parts[w], sm_row[w], sm_skip[w] > 0);
    }
  }
}

// The merge after the kernel for few rows: block c looks at the border between the runs of CTAs
// c - 1 and c.  If it lies inside an item, that item's partials are those of the CTAs whose
// runs reach into it, and the blocks of all its borders share its rows.
template <int D, bool SHARED>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
    chunk_runs_merge_kernel(const __grid_constant__ ChunkArgs a, const float* part_o, const float* part_lse) {
  __shared__ BlockJoin<D> sm_join;
  // (the second pass of a shared prefix may start)
  if constexpr (SHARED) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x + 1;
  ChunkRuns<SHARED> runs;
  ChunkShare sh;
  // (reads lengths only, which were there before the attention kernel; its CTAs start as those of that
  // kernel leave)
  const bool any = chunk_find_runs<32 * kRowsPerBlock, SHARED>(a, a.n_wave, c, &runs, &sh);
  const int tile = any ? runs.s : 0;
  // the attention kernel before it on the stream is complete and its writes are visible (also where
  // there is nothing to do: what comes after this grid may rely on both)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tile == 0) return;
  const int64_t u0 = sh.start(c) - tile;  // the item's first tile
  const int c0 = sh.owner(u0), c1 = sh.owner(u0 + runs.kt - 1);
  const int k = c1 - c0 + 1, borders = c1 - c0, mine = c - c0 - 1;
  const int first = sh.start(c0) == u0 ? 2 * c0 : 2 * c0 + 1;  // c0's run begins with the item, or ends in it
  const int g = runs.g, m0 = runs.mt * a.rows, rows = min(a.rows, runs.n * a.G - m0);
  auto out_row = [&](int r) -> int64_t {
    const int m = m0 + r;
    return (static_cast<int64_t>(runs.row0) + m / a.G) * (a.Hkv * a.G) + g * a.G + m % a.G;
  };
  auto at = [&](int r) {
    const int64_t p0 = static_cast<int64_t>(first) * a.rows + r, p1 = static_cast<int64_t>(2 * c0) * a.rows + r;
    const int64_t step = 2 * a.rows;
    return [p0, p1, step](int i) -> int64_t { return i == 0 ? p0 : p1 + i * step; };
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (k <= kWarpParts) {
    for (int r = mine * kRowsPerBlock + warp; r < rows; r += borders * kRowsPerBlock)
      store_row<D, SHARED>(a, out_row(r), join<D>(part_o, part_lse, at(r), 0, 1, k, lane), lane, runs.skip > 0);
  } else {
    for (int r = mine; r < rows; r += borders)
      join_by_block<D, SHARED>(a, sm_join, part_o, part_lse, at(r), k, out_row(r), runs.skip > 0);
  }
}

constexpr int kPlanThreads = 512;

// The plan of a call, for the persistent attention kernel and the merge after it.  One block:
// two loads and two scans a sequence, a few microseconds, under which the next grid starts.
template <bool SHARED>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a pass of a shared prefix: the groups' arrays are there, and the pass before has left the workspace
  if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t sm_scan[2 * (kPlanThreads / 32)];
  int64_t items, merged;
  chunk_make_plan<kPlanThreads, SHARED>(a, sm_scan, &items, &merged,
                                [&](int b, int first, int rt, int k, int part_row, int merge_row) {
                                  chunk_write_plan(a, b, first, rt, k, part_row, merge_row);
                                });
  if (threadIdx.x == 0) {
    a.plan[kPlanItems] = static_cast<int>(items);
    a.plan[kPlanMerged] = static_cast<int>(merged);
    a.plan[kPlanNext] = 0;
  }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t stream) {
  if (a.shared) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_plan_kernel<true>, a);
  }
  chunk_plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_chunk_runs_merge(const ChunkArgs& a, int32_t d, const float* part_o, const float* part_lse,
                                    cudaStream_t stream) {
  if (a.n_wave <= 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(a.n_wave - 1));
  cfg.blockDim = dim3(32 * kRowsPerBlock);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = d == 64 ? (a.shared ? chunk_runs_merge_kernel<64, true> : chunk_runs_merge_kernel<64, false>)
                              : (a.shared ? chunk_runs_merge_kernel<128, true> : chunk_runs_merge_kernel<128, false>);
  return cudaLaunchKernelEx(&cfg, kernel, a, part_o, part_lse);
}

cudaError_t launch_chunk_merge(const ChunkArgs& a, int32_t d, const float* part_o, const float* part_lse,
                               int64_t max_rows, cudaStream_t stream) {
  if (max_rows <= 0) return cudaSuccess;
  // programmatic dependent launch, as the merge of equal splits (merge_lse.cu)
  cudaLaunchConfig_t cfg = {};
  // blocks beyond a few waves would only find the row count already passed
  const int64_t blocks = (max_rows + kRowsPerBlock - 1) / kRowsPerBlock;
  cfg.gridDim = dim3(static_cast<unsigned int>(blocks < 1216 ? blocks : 1216));
  cfg.blockDim = dim3(32 * kRowsPerBlock);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = d == 64 ? (a.shared ? chunk_merge_kernel<64, true> : chunk_merge_kernel<64, false>)
                              : (a.shared ? chunk_merge_kernel<128, true> : chunk_merge_kernel<128, false>);
  return cudaLaunchKernelEx(&cfg, kernel, a, part_o, part_lse);
}

}  // namespace skv
