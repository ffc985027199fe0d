// The groups of attn_shared_prefix_paged: sequences whose first block-table entries are the same pages.
//
// Attention over [0, P) and over [P, p] joins exactly (out = sum w_i o_i / sum w_i, w_i = exp(lse_i)), so
// the prefix is attended once for all rows of a group, as one sequence that every row sees whole (its
// pages are read once, and the rows of all sequences fill the tensor cores' tiles together), and
// the rest of every sequence by itself; the second pass joins its rows with the first one's.
//
// This kernel says what is shared: a prefix is cut to whole tiles of kTileN tokens, and to tokens that
// every new token of the group sees (before the first new token of each of its sequences), so that
// whatever lengths it is given, a sequence's own pass covers the rest.  One block a group, and one for
// the sequences of no group; a few loads a sequence.
//
// Measured: 64 sequences of 100 to 1000 tokens behind one document of 32768, 64 / 8 heads, one token each: 115 us
// where attn_chunk_paged over the same pages takes 630 to 670 (more than half of its reads come from L2: HBM alone would
// take 1290); 58 of the 115 the tensor cores over the prefix (29 tiles a CTA of 1.4 us), 10 its merge, 36 the rest of
// the sequences.  The five launches and the second pass's starts cost 10 to 30 us, which about 2^20 (sequence, KV head,
// prefix token) win back: 16 sequences behind 2048 tokens, 8 KV heads, 45 us against 30, behind 8192 49 against 55.
#include <cuda_runtime.h>

#include <climits>

#include "skv_internal.h"

namespace skv {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) shared_groups_kernel(const __grid_constant__ SharedArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the next kernel sets itself up meanwhile)
  __shared__ int sm_len[kThreads / 32], sm_first[kThreads / 32];
  const int j = blockIdx.x;
  auto bound = [&](int i) { return min(max(__ldg(a.cu_groups + i), 0), a.B); };
  auto row_of = [&](int b) { return min(max(__ldg(a.cu_q + b), 0), a.T); };
  if (j == a.n_groups) {
    const int lo = bound(0), hi = bound(a.n_groups);
    for (int b = threadIdx.x; b < a.B; b += kThreads)
      if (b < lo || b >= hi) a.skip[b] = 0;
    return;
  }
  const int b0 = bound(j), b1 = bound(j + 1);
  // tokens before the new ones of every sequence that has some, and the first such sequence
  int len = min(max(__ldg(a.prefix_lens + j), 0), a.cap), first = INT_MAX;
  for (int b = b0 + threadIdx.x; b < b1; b += kThreads) {
    const int n = row_of(b + 1) - row_of(b);
    if (n > 0) {
      len = min(len, max(__ldg(a.seq_lens + b), 0) - n);
      first = min(first, b);
    }
  }
  len = __reduce_min_sync(0xffffffffu, len);
  first = __reduce_min_sync(0xffffffffu, first);
  if ((threadIdx.x & 31) == 0) {
    sm_len[threadIdx.x >> 5] = len;
    sm_first[threadIdx.x >> 5] = first;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    len = min(len, sm_len[w]);
    first = min(first, sm_first[w]);
  }
  len = first == INT_MAX ? 0 : max(len, 0) / kTileN * kTileN;
  for (int b = b0 + threadIdx.x; b < b1; b += kThreads) a.skip[b] = len;
  if (threadIdx.x == 0) {
    a.group_len[j] = len;
    a.table_row[j] = min(first, a.B - 1);
    a.group_rows_at[j] = row_of(b0);
    if (j == a.n_groups - 1) a.group_rows_at[a.n_groups] = row_of(b1);
  }
}

}  // namespace

cudaError_t launch_shared_groups(const SharedArgs& a, cudaStream_t stream) {
  shared_groups_kernel<<<a.n_groups + 1, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace skv
