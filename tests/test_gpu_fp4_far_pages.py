"""4-bit pages whose codes lie past 2^34 bytes and whose block scales past 2^31: what is written there, read back and
attended is what the same pages give as a small cache, bit for bit."""

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
N, Hkv, L, Hq = (1 << 19) + 100, 8, 64, 16


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_far_pages():
    torch.cuda.empty_cache()
    g = torch.Generator().manual_seed(41)
    far = [torch.empty(N, Hkv, L, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    far += [torch.empty(N, Hkv, L, 8, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    # the first two pages are shared, the lengths end inside a page
    table = ints([N - 1, N // 2 + 5, 3, N - 70, N // 4 * 3], [N - 1, N // 2 + 5, N - 9, 7, N // 3])
    lens = ints(300, 268)
    k_new = []
    for b, (first, m) in enumerate(((0, 300), (128, 268))):
        qkv = torch.randn(m - first, (Hq + 2 * Hkv) * 128, generator=g).bfloat16().to(DEV)
        q, k, v = paged.split_qkv(qkv, Hq, Hkv)
        skv.qk_norm_rope_append(q, k, v, far[0], far[1], ints(m), ints(0, m - first), table[b:b + 1].contiguous(),
                                k_scale=far[2], v_scale=far[3])
        k_new.append(k.cpu().double())
    used = sorted(set(table.flatten().tolist()))
    at = torch.tensor(used, device=DEV)
    near = [x.view(torch.uint8)[at].view(x.dtype) for x in far]
    near_table = ints(*[[used.index(p) for p in row] for row in table.tolist()])
    caches = ((far, table), (near, near_table))
    # what was written is the new tokens' keys, off by half a step of e2m1 at most: 1 / 6 of the block's largest
    page, row = near_table[0].cpu().long()[torch.arange(300) // L], torch.arange(300) % L
    got = (F.values_of(near[0]) * F.scales_of(near[2]).repeat_interleave(F.BLOCK, -1))[page, :, row]
    most = k_new[0].unflatten(-1, (-1, F.BLOCK)).abs().amax(-1, keepdim=True)
    off = (got - k_new[0]).unflatten(-1, (-1, F.BLOCK)).abs()
    # (the scale's own rounding moves the values by 2^-4 of themselves, and saturates the largest by as much)
    assert (off <= (1 / 6 + 2.0 ** -4) * most * (1 + 2.0 ** -4)).all()

    def same(call):
        a, b = (call(*c) for c in caches)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert torch.isfinite(x).all() and torch.equal(x, y)

    same(lambda p, t: skv.kv_read_paged(p[0], p[1], ints(0, 300, 568), t, n_tokens=568, k_scale=p[2], v_scale=p[3]))
    for n in (1, 2, 3, 40):  # with the bounds: 8 rows of a KV head, 16 or 32, and the tensor cores
        q = torch.randn(2 * n, Hq, 128, generator=g).bfloat16().to(DEV)
        for bound in (n, 12, None):
            same(lambda p, t: skv.attn_chunk_paged(q, p[0], p[1], lens, ints(0, n, 2 * n), t, max_q_len=bound, k_scale=p[2],
                                                   v_scale=p[3]))
            same(lambda p, t: skv.attn_shared_prefix_paged(q, p[0], p[1], lens, ints(0, n, 2 * n), t, ints(0, 2), ints(128),
                                                           max_q_len=bound, k_scale=p[2], v_scale=p[3]))
    assert skv.device_error() == 0
    del far, caches
    torch.cuda.empty_cache()
