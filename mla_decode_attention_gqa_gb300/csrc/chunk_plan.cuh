// Work decomposition of attention over ragged chunks of new tokens (attn_chunk_paged), done
// on the device: the host knows T packed rows and B sequences, never their lengths, so one
// call can be captured into a graph and replayed with other lengths.
//
// Sequence b has n = cu_q[b+1] - cu_q[b] new tokens, the last n of its m = seq_lens[b] cached
// ones; row i sits at position m - n + i.  Its rows of one KV head (n times the group's G, or G
// padded to a power of two) are cut into row tiles of R rows.  For the tensor-core kernel every row
// tile's KV tiles are cut into k_b chunks:
//   W   = sum over b of (row tiles) * Hkv * (KV tiles of its last row tile)
//   L   = max(1, ceil(W / n_target)),  k_b = max(1, floor((KV tiles) / L))
// so the work items with k_b > 1 are at most W / L <= n_target, whatever the lengths are
// (which bounds the workspace), and those with k_b = 1 at most Hkv * (row tiles).
//
// The persistent tensor-core kernel takes its items from a plan that one small kernel wrote
// before it.  The kernel for few rows cuts the work into equal runs instead, which every CTA
// finds with a scan of its own over the sequences (one pass of loads when B is at most the block's
// threads).
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
  int skip;      // of those, the first ones that another pass attends
  int part_row;  // first partial row of the sequence (n_chunk > 1)
};

// SHARED: a pass of a shared prefix, with the arrays that ChunkArgs lists for it.  A template argument
// throughout, so that the other calls carry nothing of it (as tests of the arguments it took a call
// of one token 1.5 us of 17, a windowed prompt 4 of 275).
// (Those arrays are written by a kernel before, so they are not read through the read-only path.)
template <bool SHARED>
__device__ __forceinline__ void chunk_lengths(const ChunkArgs& a, int b, int* row0, int* n, int* m, int* skip) {
  int lo, hi, len;
  if (SHARED && a.group_rows_at) {
    lo = __ldcg(a.group_rows_at + b), hi = __ldcg(a.group_rows_at + b + 1);
    len = __ldcg(a.seq_lens + b);
  } else {
    lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1);
    len = __ldg(a.seq_lens + b);
  }
  lo = min(max(lo, 0), a.T), hi = min(max(hi, 0), a.T);
  *row0 = lo;
  *n = max(hi - lo, 0);
  *m = max(len, 0);
  *skip = 0;
  if constexpr (SHARED) {
    if (a.whole && *m == 0) *n = 0;  // (nothing to do for a group without a prefix)
    if (a.skip) *skip = __ldcg(a.skip + b);
  }
}

// Position of the first of n new tokens, and from each to the next.
template <bool SHARED>
__device__ __forceinline__ int chunk_pos0(const ChunkArgs& a, int n, int m) {
  return SHARED && a.whole ? m - 1 : m - n;
}
template <bool SHARED>
__device__ __forceinline__ int chunk_pos_step(const ChunkArgs& a) {
  return SHARED && a.whole ? 0 : 1;
}

// A row's result over its own tokens (out, lse) joined with the one over its prefix: the weights of the
// two, and the lse of both.  A part that saw nothing weighs nothing; a NaN on either side stays, also beside a
// part of -inf, where fmaxf would drop it.  (Both rows are multiplied by their weights, zero or not: 0 times a NaN or
// an infinity, that of a value which a softmax over all tokens would have multiplied by 0 as well, is NaN.)
struct ChunkJoin {
  float own, prior, lse;
};
__device__ __forceinline__ ChunkJoin chunk_join(float lse, float prior_lse) {
  const float m = fmaxf(lse, prior_lse);
  ChunkJoin j;
  if (lse != lse || prior_lse != prior_lse) {
    j.own = j.prior = j.lse = __int_as_float(0x7fc00000);
    return j;
  }
  if (m == -INFINITY) {
    j.own = j.prior = 0.f;
    j.lse = -INFINITY;
    return j;
  }
  const float a = __expf(lse - m), b = __expf(prior_lse - m), sum = a + b;
  j.own = a / sum;
  j.prior = b / sum;
  j.lse = m + logf(sum);
  return j;
}

// Page of token `tok` of sequence (or group) b.
template <bool SHARED>
__device__ __forceinline__ int chunk_page_of(const PartialParams& p, int b, int tok) {
  return kv_page_of(p, SHARED && p.ck.table_row ? __ldcg(p.ck.table_row + b) : b, tok);
}

// Blocks of kTileN tokens seen by the rows at positions [p0, p1] of a sequence with `cap` tokens
// at most: those below n_first hold the sinks, then come the ones from win on; block i of the
// item is i < n_first ? i : win + (i - n_first).  lo / hi: the window's token range (of all
// the rows together); sinks: the first tokens seen besides it.
struct ChunkTiles {
  int lo, hi, sinks;
  int n_first, win, n;
};

__device__ __forceinline__ ChunkTiles chunk_tiles(int window, int n_sink, int cap, int skip, int p0, int p1) {
  constexpr int tile = kTileN;
  ChunkTiles t;
  t.hi = min(max(p1 + 1, 0), cap);
  t.lo = (window > 0 && p0 >= window) ? p0 - window + 1 : skip;  // (a call with skips has no window)
  t.sinks = min(n_sink, t.hi);
  if (t.sinks >= t.lo) t.lo = 0;  // the sinks reach the window: one range
  t.n_first = t.lo > 0 ? (t.sinks + tile - 1) / tile : 0;
  const int end = (t.hi + tile - 1) / tile;
  t.win = min(t.lo / tile, end);  // (all rows far behind the last token: no block past the last one)
  if (t.lo > 0 && t.n_first > t.win) t.n_first = t.win;  // a block of both is the window's
  t.n = t.n_first + max(end - t.win, 0);
  return t;
}

// Row tiles per KV head, and KV tiles of the row tile that has most: the last one; with a window, an
// earlier one may touch a block more than the last, so there the bound is of their length alone.
template <bool SHARED>
__device__ __forceinline__ void chunk_extent(const ChunkArgs& a, int n, int m, int skip, int* row_tiles, int* kv_tiles) {
  *row_tiles = static_cast<int>((static_cast<int64_t>(n) * a.group_rows + a.rows - 1) / a.rows);
  const int span = min(n, (a.rows + a.group_rows - 1) / a.group_rows + 1);
  const ChunkTiles t = chunk_tiles(a.window, a.n_sink, a.cap, skip, SHARED && a.whole ? m - 1 : m - span, m - 1);
  int blocks = t.n;
  if (a.window > 0 && *row_tiles > 1) {
    const int64_t seen = static_cast<int64_t>(a.window) - 1 + span;  // tokens of a row tile's window
    const int64_t most = (seen + 2 * kTileN - 2) / kTileN + (a.n_sink + static_cast<int64_t>(kTileN) - 1) / kTileN;
    blocks = static_cast<int>(min(most, (static_cast<int64_t>(t.hi) + kTileN - 1) / kTileN));
  }
  const int per = a.tile / kTileN;
  *kv_tiles = max((blocks + per - 1) / per, 1);
}

// The plan in device memory: [kPlanItems] work items, [kPlanMerged] rows to merge, [kPlanNext] the
// next item to hand out, and for each sequence its first item, first row to merge, first partial
// row, row tiles and chunks per row tile.
__device__ __forceinline__ void chunk_write_plan(const ChunkArgs& a, int b, int first, int rt, int k, int part_row,
                                                 int merge_row) {
  int32_t* e = a.plan + kPlanHead + static_cast<int64_t>(kPlanRow) * b;
  e[0] = first;
  e[1] = merge_row;
  e[2] = part_row;
  e[3] = rt;
  e[4] = k;
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

// The plan of one call, computed by all NT threads of a block: `visit(b, first item, row tiles,
// chunks, first partial row, first row to merge)` for every sequence, totals in *items and
// *merged.  A visitor must not synchronise.
template <int NT, bool SHARED, class F>
__device__ __forceinline__ void chunk_make_plan(const ChunkArgs& a, int64_t* sm_scan, int64_t* items, int64_t* merged,
                                                F&& visit) {
  const int tid = threadIdx.x;
  int64_t w = 0, zero = 0, total, unused;
  for (int b = tid; b < a.B; b += NT) {
    int row0, n, m, skip, rt, kt;
    chunk_lengths<SHARED>(a, b, &row0, &n, &m, &skip);
    chunk_extent<SHARED>(a, n, m, skip, &rt, &kt);
    w += static_cast<int64_t>(rt) * a.Hkv * kt;
  }
  chunk_block_scan<NT>(w, zero, &total, &unused, sm_scan);
  // (prefixes: one wave of items, with chunks rounded to the nearest number instead of down, since every one
  // writes fp32 rows that the merge reads again; 4/3 of W / L at most.  64 rows of 64 / 8 heads behind 32768
  // tokens: 9 chunks a row tile where four waves made 36, 60 us and 8 of merge for 81 and 27)
  const bool whole = SHARED && a.whole;
  const int64_t target = whole || total <= a.n_wave * static_cast<int64_t>(kChunkShortTiles) ? a.n_wave : a.n_target;
  const int L = static_cast<int>(min(max((total + target - 1) / target, (int64_t)1), (int64_t)1 << 30));
  const int Hq = a.Hkv * a.G;
  int64_t it0 = 0, part0 = 0, mr0 = 0;  // of the sequences before this pass
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + tid;
    int row0 = 0, n = 0, m = 0, skip = 0, rt = 0, kt = 1, k = 1;
    if (b < a.B) {
      chunk_lengths<SHARED>(a, b, &row0, &n, &m, &skip);
      chunk_extent<SHARED>(a, n, m, skip, &rt, &kt);
      k = max(1, static_cast<int>((kt + (whole ? static_cast<int64_t>(L / 2) : 0)) / L));
    }
    const int64_t mine = static_cast<int64_t>(rt) * a.Hkv * k;
    const int64_t rows = k > 1 ? static_cast<int64_t>(n) * Hq : 0;
    int64_t x = mine, y = rows * k, z = rows, tx, ty, tz;
    chunk_block_scan<NT>(x, y, &tx, &ty, sm_scan);
    chunk_block_scan<NT>(z, zero, &tz, &unused, sm_scan);
    if (b < a.B)
      visit(b, static_cast<int>(it0 + x - mine), rt, k, static_cast<int>(part0 + y - rows * k),
            static_cast<int>(mr0 + z - rows));
    it0 += tx;
    part0 += ty;
    mr0 += tz;
    zero = 0;
  }
  *items = it0;
  *merged = mr0;
}

// Item number r of sequence b: later row tiles (which see more) first; a row tile's chunks and
// heads side by side.
template <bool SHARED>
__device__ __forceinline__ ChunkItem chunk_item_of(const ChunkArgs& a, int b, int r, int rt, int k, int part_row) {
  ChunkItem it;
  it.b = b;
  chunk_lengths<SHARED>(a, b, &it.row0, &it.n, &it.m, &it.skip);
  it.n_chunk = k;
  it.part_row = part_row;
  it.c = r % k;
  r /= k;
  it.g = r % a.Hkv;
  it.mt = rt - 1 - r / a.Hkv;
  return it;
}

// Work item `idx` from the written plan (idx < its number of items).  Warp-collective: a
// 32-way search for the last sequence whose first item is <= idx (sequences without items
// share the first item of the one after them).
template <bool SHARED>
__device__ __forceinline__ ChunkItem chunk_item_at(const ChunkArgs& a, int idx) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool before = lane * step < n && __ldcg(a.plan + kPlanHead + static_cast<int64_t>(kPlanRow) * b) <= idx;
    const int hits = __popc(__ballot_sync(0xffffffffu, before));  // >= 1: a prefix of the lanes
    const int skip = max(hits - 1, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  const int32_t* e = a.plan + kPlanHead + static_cast<int64_t>(kPlanRow) * lo;
  return chunk_item_of<SHARED>(a, lo, idx - __ldcg(e), __ldcg(e + 3), __ldcg(e + 4), __ldcg(e + 2));
}

// ---- equal runs (the kernel for few rows): all items' KV tiles in one line -- sequence after
// sequence, in each the items (row tile, KV head), in each its tiles -- cut into n equal runs.  An
// item counts `start` tiles more than it has, ahead of them: what its rows' loads and the
// join of the warps take (without, a CTA with many short items took half as long again).

// How U tiles are shared by n CTAs: the first r take q + 1, the others q.
struct ChunkShare {
  int64_t q;
  int r, n;
  __device__ __forceinline__ int64_t start(int c) const { return q * c + min(c, r); }
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t head = (q + 1) * r;
    return static_cast<int>(u < head ? u / (q + 1) : r + (u - head) / q);
  }
};

// The part of one item that lies in a run.
struct ChunkPiece {
  int b, g, mt;
  int row0, n, m;   // first packed row, new tokens, cached tokens with them
  int skip;         // of those, the first ones that another pass attends
  ChunkTiles tl;
  int i0, n_tiles;  // its blocks in tl's run
  int slot;         // the partial's number, two of each CTA; < 0: the whole item, final
  __device__ __forceinline__ int token(int i) const {  // first token of tile i
    const int x = i0 + i;
    return (x < tl.n_first ? x : tl.win + (x - tl.n_first)) * kTileN;
  }
};

// A CTA's run, piece by piece.  (The divisions are done once, by find: a piece begins where the one
// before ends.)
template <bool SHARED>
struct ChunkRuns {
  int64_t left;  // tiles left
  int cta, b, row0, n, m, skip, rt, kt;  // kt: with the start
  int g, mt, s;  // the next piece's item, and its first tile there
  bool head;
  __device__ __forceinline__ void load(const ChunkArgs& a) {
    chunk_lengths<SHARED>(a, b, &row0, &n, &m, &skip);
    chunk_extent<SHARED>(a, n, m, skip, &rt, &kt);
    kt += a.start;
  }
  // Tiles [at, at + count) of those from sequence `seq` on (which holds the first of them).
  __device__ __forceinline__ void find(const ChunkArgs& a, int c, int seq, int64_t at, int64_t count) {
    cta = c;
    b = seq;
    left = count;
    head = true;
    load(a);
    const int64_t item = at / kt;
    s = static_cast<int>(at - item * kt);
    const int r = static_cast<int>(item / a.Hkv);
    g = static_cast<int>(item - static_cast<int64_t>(r) * a.Hkv);
    mt = rt - 1 - r;
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, ChunkPiece* pc) {
    if (left <= 0) return false;
    while (mt < 0) {  // (tiles are left: there is such a sequence)
      ++b;
      load(a);
      mt = rt - 1;
    }
    const int e = static_cast<int>(min(static_cast<int64_t>(kt), s + left));
    pc->b = b, pc->row0 = row0, pc->n = n, pc->m = m, pc->skip = skip;
    pc->mt = mt;
    pc->g = g;
    const int m0 = mt * a.rows, m_last = min(m0 + a.rows, n * a.group_rows) - 1;
    const int pos0 = chunk_pos0<SHARED>(a, n, m), step = chunk_pos_step<SHARED>(a);
    pc->tl = chunk_tiles(a.window, a.n_sink, a.cap, skip, pos0 + m0 / a.group_rows * step, pos0 + m_last / a.group_rows * step);
    pc->i0 = min(max(s - a.start, 0), pc->tl.n);
    pc->n_tiles = min(max(e - a.start, 0), pc->tl.n) - pc->i0;  // (an earlier row tile may see fewer than kt)
    pc->slot = (s == 0 && e == kt) ? -1 : 2 * cta + (head ? 0 : 1);
    head = false;
    left -= e - s;
    s = 0;
    if (++g == a.Hkv) g = 0, --mt;
    return true;
  }
};

// Run `cta` of at most n_cta; false if there is none.  Every thread of the block calls it.
template <int NT, bool SHARED>
__device__ __forceinline__ bool chunk_find_runs(const ChunkArgs& a, int n_cta, int cta, ChunkRuns<SHARED>* runs,
                                                ChunkShare* share = nullptr) {
  __shared__ int64_t sm_scan[2 * (NT / 32)];
  __shared__ int64_t sm_first;
  __shared__ int sm_b;
  const int tid = threadIdx.x;
  int64_t w = 0, zero = 0, total, unused;
  for (int b = tid; b < a.B; b += NT) {
    int row0, n, m, skip, rt, kt;
    chunk_lengths<SHARED>(a, b, &row0, &n, &m, &skip);
    chunk_extent<SHARED>(a, n, m, skip, &rt, &kt);
    w += static_cast<int64_t>(rt) * a.Hkv * (kt + a.start);
  }
  chunk_block_scan<NT>(w, zero, &total, &unused, sm_scan);
  ChunkShare sh;
  sh.n = static_cast<int>(min(static_cast<int64_t>(n_cta), max(total / kChunkMinTiles, (int64_t)1)));
  sh.q = total / sh.n;
  sh.r = static_cast<int>(total % sh.n);
  if (share) *share = sh;
  if (cta >= sh.n || total == 0) return false;  // uniform in the block
  const int64_t u = sh.start(cta);
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B && before <= u; b0 += NT) {  // uniform in the block
    const int b = b0 + tid;
    int row0, n, m, skip, rt = 0, kt = 1;
    if (b < a.B) {
      chunk_lengths<SHARED>(a, b, &row0, &n, &m, &skip);
      chunk_extent<SHARED>(a, n, m, skip, &rt, &kt);
    }
    const int64_t mine = static_cast<int64_t>(rt) * a.Hkv * (kt + a.start);
    int64_t x = mine, y = 0, tx, ty;
    chunk_block_scan<NT>(x, y, &tx, &ty, sm_scan);
    const int64_t first = before + x - mine;
    if (b < a.B && u >= first && u < first + mine) {
      sm_first = first;
      sm_b = b;
    }
    before += tx;
  }
  __syncthreads();
  runs->find(a, cta, sm_b, u - sm_first, sh.start(cta + 1) - u);
  return true;
}

#endif  // __CUDACC__

}  // namespace skv
