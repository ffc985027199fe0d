// Work decomposition of attention over ragged chunks of new tokens (attn_chunk_paged), done
// on the device: the host knows T packed rows and B sequences, never their lengths, so one
// call can be captured into a graph and replayed with other lengths.
//
// Sequence b has n = cu_q[b+1] - cu_q[b] new tokens, the last n of its m = seq_lens[b] cached
// ones; row i sits at position m - n + i.  Its rows of one KV head (n times the
// group's G, or G padded to a power of two) are cut into row tiles of R rows, and every row tile's KV tiles into k_b chunks:
//   W   = sum over b of (row tiles) * Hkv * (KV tiles of its last row tile)
//   L   = max(1, ceil(W / n_target)),  k_b = max(1, floor((KV tiles) / L))
// so the work items with k_b > 1 are at most W / L <= n_target, whatever the lengths are
// (which bounds the workspace), and those with k_b = 1 at most Hkv * (row tiles).  Every
// block finds its own item with one scan over the sequences (one pass of loads when B is at
// most the block's threads), which costs less than a launch that would write a plan.
#pragma once

#include "skv_internal.h"

namespace skv {

#ifdef __CUDACC__

// One block's work item, and the sequence's numbers the kernels need.
struct ChunkItem {
  int b;         // sequence
  int g;         // KV head
  int mt;        // row tile
  int c;         // chunk of the row tile's KV tiles
  int n_chunk;   // chunks per row tile of this sequence (1: the block writes the final rows)
  int row0;      // first packed row (cu_q[b])
  int n;         // new tokens
  int m;         // cached tokens with them
  int part_row;  // first partial row of the sequence (n_chunk > 1)
};

__device__ __forceinline__ void chunk_lengths(const ChunkArgs& a, int b, int* row0, int* n, int* m) {
  const int lo = min(max(__ldg(a.cu_q + b), 0), a.T), hi = min(max(__ldg(a.cu_q + b + 1), 0), a.T);
  *row0 = lo;
  *n = max(hi - lo, 0);
  *m = __ldg(a.seq_lens + b);
}

// Token tiles seen by the rows at positions [p0, p1] of a sequence with `cap` tokens at most:
// the tiles below n_first hold the sinks, then come the tiles from win on; tile i of the
// item is i < n_first ? i : win + (i - n_first).  lo / hi: the window's token range (of all
// the rows together); sinks: the first tokens seen besides it.
struct ChunkTiles {
  int lo, hi, sinks;
  int n_first, win, n;
};

__device__ __forceinline__ ChunkTiles chunk_tiles(int window, int n_sink, int cap, int p0, int p1, int tile) {
  ChunkTiles t;
  t.hi = min(max(p1 + 1, 0), cap);
  t.lo = (window > 0 && p0 >= window) ? p0 - window + 1 : 0;
  t.sinks = min(n_sink, t.hi);
  if (t.sinks >= t.lo) t.lo = 0;  // the sinks reach the window: one range
  t.n_first = t.lo > 0 ? (t.sinks + tile - 1) / tile : 0;
  t.win = t.lo / tile;
  const int end = (t.hi + tile - 1) / tile;
  if (t.lo > 0 && t.n_first > t.win) t.n_first = t.win;  // a tile of both is the window's
  t.n = t.n_first + max(end - t.win, 0);
  return t;
}

// Row tiles per KV head and KV tiles of the last row tile (an upper bound of the others').
__device__ __forceinline__ void chunk_extent(const ChunkArgs& a, int n, int m, int* row_tiles, int* kv_tiles) {
  *row_tiles = static_cast<int>((static_cast<int64_t>(n) * a.group_rows + a.rows - 1) / a.rows);
  const int span = min(n, (a.rows + a.group_rows - 1) / a.group_rows + 1);
  const ChunkTiles t = chunk_tiles(a.window, a.n_sink, a.cap, m - span, m - 1, a.tile);
  *kv_tiles = max(t.n, 1);
}

// Inclusive sums over the block's threads of x and y; total of both in *tx, *ty.
template <int NT>
__device__ __forceinline__ void chunk_block_scan(int64_t& x, int64_t& y, int64_t* tx, int64_t* ty, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += ux;
      y += uy;
    }
  }
  __syncthreads();  // the scratch's earlier readers are done
  if (lane == 31) {
    sm[2 * warp] = x;
    sm[2 * warp + 1] = y;
  }
  __syncthreads();
  int64_t bx = 0, by = 0, sx = 0, sy = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int64_t vx = sm[2 * w], vy = sm[2 * w + 1];
    if (w < warp) {
      bx += vx;
      by += vy;
    }
    sx += vx;
    sy += vy;
  }
  x += bx;
  y += by;
  *tx = sx;
  *ty = sy;
}

// The block's work item; false if there are fewer items than blocks.  Block 0 also writes the
// merge's table (see chunk_merge.cu).  Every thread of the block calls it.
template <int NT>
__device__ __forceinline__ bool chunk_find_item(const ChunkArgs& a, ChunkItem* item) {
  __shared__ int64_t sm_scan[2 * (NT / 32)];
  __shared__ ChunkItem sm_item;
  __shared__ int sm_found;
  const int tid = threadIdx.x;
  if (tid == 0) sm_found = 0;
  int64_t w = 0, zero = 0, total, unused;
  for (int b = tid; b < a.B; b += NT) {
    int row0, n, m, rt, kt;
    chunk_lengths(a, b, &row0, &n, &m);
    chunk_extent(a, n, m, &rt, &kt);
    w += static_cast<int64_t>(rt) * a.Hkv * kt;
  }
  chunk_block_scan<NT>(w, zero, &total, &unused, sm_scan);
  const int64_t target = total <= a.n_wave * static_cast<int64_t>(kChunkShortTiles) ? a.n_wave : a.n_target;
  const int L = static_cast<int>(min(max((total + target - 1) / target, (int64_t)1), (int64_t)1 << 30));

  const bool writes_plan = blockIdx.x == 0 && a.plan != nullptr;
  const int Hq = a.Hkv * a.G;
  int64_t items = 0, parts = 0;  // of the sequences before this pass
  int64_t merged = 0;            // rows to merge of the sequences before this pass
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + tid;
    int row0 = 0, n = 0, m = 0, rt = 0, kt = 1, k = 1;
    if (b < a.B) {
      chunk_lengths(a, b, &row0, &n, &m);
      chunk_extent(a, n, m, &rt, &kt);
      k = max(1, kt / L);
    }
    const int64_t mine = static_cast<int64_t>(rt) * a.Hkv * k;
    const int64_t my_rows = k > 1 ? static_cast<int64_t>(n) * Hq : 0;
    int64_t x = mine, y = my_rows * k, tx, ty;
    chunk_block_scan<NT>(x, y, &tx, &ty, sm_scan);
    const int64_t first = items + x - mine, part0 = parts + y - my_rows * k;
    if (b < a.B && blockIdx.x >= first && blockIdx.x < first + mine) {
      int r = static_cast<int>(blockIdx.x - first);
      ChunkItem it;
      it.b = b;
      it.n_chunk = k;
      it.row0 = row0;
      it.n = n;
      it.m = m;
      it.part_row = static_cast<int>(part0);
      // later row tiles (which see more) first; a row tile's chunks and heads side by side
      it.c = r % k;
      r /= k;
      it.g = r % a.Hkv;
      it.mt = rt - 1 - r / a.Hkv;
      sm_item = it;
      sm_found = 1;
    }
    if (writes_plan) {  // uniform in the block
      int64_t mx = my_rows, my = 0, tmx, tmy;
      chunk_block_scan<NT>(mx, my, &tmx, &tmy, sm_scan);
      if (b < a.B) {
        a.plan[3 * b] = static_cast<int>(merged + mx - my_rows);  // first row to merge
        a.plan[3 * b + 1] = static_cast<int>(part0);              // first partial row
        a.plan[3 * b + 2] = k;
      }
      merged += tmx;
    }
    items += tx;
    parts += ty;
    if (!writes_plan && blockIdx.x < items) break;  // uniform in the block
  }
  if (writes_plan && tid == 0) a.plan[3 * a.B] = static_cast<int>(merged);
  __syncthreads();
  *item = sm_item;
  return sm_found != 0;
}

#endif  // __CUDACC__

}  // namespace skv
