"""GPU tests of attn_chunk_paged's edges on each of its kernels: the one for 16 rows of a KV head, the
one for 32, and the tensor cores.  The bound on the chunk lengths chooses the kernel; ``bound``
asserts the rule, so that a case cannot move to another kernel unseen."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from tests import chunk_ref as R
from tests.test_gpu_chunk_fp8 import KERNELS, WEIGHT, bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [("bf16", 64), ("bf16", 128), ("fp8", 128)]


def run(c, kernel, window=0, n_sink=0, **kw):
    q = kw.pop("q", c["q"])
    out, lse = skv.attn_chunk_paged(q, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=bound(kernel, q.shape[1] // c["k_pages"].shape[1], q.shape[0]),
                                    window=window, n_sink=n_sink, k_scale=c["k_scale"], v_scale=c["v_scale"], **kw)
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    return out, lse


@pytest.mark.parametrize("power", [20, 28, 31, 34, 40, 60])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_scores_of_any_size(kind, d, kernel, power):
    """Queries times 2^power: all weight on the largest score wherever that is told from the next, in
    one piece and in several (solo and pair items on the tensor cores)."""
    c = R.make_case([12, 70, 1], [700, 330, 2000], 8, 2, d, fp8=kind == "fp8", seed=power, device=DEV)
    c["q"] = (c["q"].float() * 2.0 ** power).to(torch.bfloat16)
    out, lse = (x.cpu().double() for x in run(c, kernel))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    ro, rl, size = R.attend(c)
    # a score: 128 additions off by 2^-23 of the terms' sum, below 16 * 2^power; fp8: a query's part below
    # 2^-17 of its largest may be lost, 4e-4 * 2^power; both below 2^(power - 10) together
    off = 2.0 ** (power - 10)
    assert (lse - rl).abs().max() <= off
    # rows whose largest score stands out by 4 of that: the others weigh exp(-2^(power - 9)), nothing
    q, clear = c["q"].cpu().double(), torch.zeros(rl.shape, dtype=torch.bool)
    k_pages, cu = R.dense(c["k_pages"], c["k_scale"]), c["cu_q"].tolist()
    for b, m in enumerate(c["seq_lens"].tolist()):
        t = torch.arange(m)
        page, at = c["block_table"][b].cpu().long()[t // 64], t % 64
        for h in range(8):
            x = q[cu[b]:cu[b + 1], h] @ k_pages[page, h // 4, at].T / math.sqrt(d)
            pos = torch.arange(m - (cu[b + 1] - cu[b]), m)
            x = x.masked_fill(t[None] > pos[:, None], -math.inf)
            top = x.topk(2, -1).values
            clear[cu[b]:cu[b + 1], h] = top[:, 0] - top[:, 1] > 4 * off
    assert clear.double().mean() > 0.5
    tol = (WEIGHT[kernel] if kind == "fp8" else 2.0 ** -8) * size + 2.0 ** -8 * ro.abs()
    assert ((out - ro).abs() <= tol)[clear].all()


# ------------------------------------------------------------------ edges, on each kernel


def check(c, kernel, window=0, n_sink=0, **kw):
    out, lse = run(c, kernel, window, n_sink, **kw)
    R.check_attention(c, out, lse, window, n_sink, kw.get("softmax_scale"), q=kw.get("q"))
    return out, lse


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_rows_that_see_nothing(kind, d, kernel):
    c = R.make_case([7, 4, 1, 3], [3, 0, 0, 64], 8, 2, d, fp8=kind == "fp8", seed=3, device=DEV)
    check(c, kernel)
    check(c, kernel, window=2, n_sink=1)
    c["seq_lens"][1] = -5
    check(c, kernel)
    c["seq_lens"][3] = 64 + 7  # one page: tokens past it do not exist
    check(c, kernel)
    check(c, kernel, window=9, n_sink=1)
    c["seq_lens"][3] = 2 ** 31 - 1  # all rows lie far behind the last token
    check(c, kernel)
    check(c, kernel, window=9, n_sink=1)
