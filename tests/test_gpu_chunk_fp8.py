"""GPU tests of attn_chunk_paged over fp8 pages where the ranges of its roundings can go wrong: V
scales that lie far apart, queries of very different size, and how many bits the weights keep.
Every case runs on the kernel for 16 rows of a KV head, on the one for 32, and on the tensor cores."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from tests import chunk_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
L = 64


def bound(kernel, G, T):
    """max_q_len that leads to a kernel for groups of G heads and T packed rows: up to 16 rows of a
    KV head, up to 32, more."""
    n = {"rows16": 16 // G, "rows32": 32 // G, "tc": T}[kernel]
    assert {"rows16": n * G <= 16, "rows32": 16 < n * G <= 32, "tc": n * G > 32}[kernel] and 1 <= n <= T
    return n


KERNELS = ["rows16", "rows32", "tc"]
WEIGHT = {"rows16": 2.0 ** -11, "rows32": 2.0 ** -11, "tc": 2.0 ** -8}  # half a step of fp16 and of bf16


def run(c, kernel, **kw):
    G, T = c["q"].shape[1] // c["k_pages"].shape[1], c["q"].shape[0]
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=bound(kernel, G, T), k_scale=c["k_scale"], v_scale=c["v_scale"], **kw)
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    return out.cpu().double(), lse.cpu().double()


def tiles_of_a_sequence(scores, spread, B, Hkv, seed):
    """B sequences of one token with G = 1: tile i of 64 tokens has scores near scores[i] (base e)
    and a V scale of 2^spread[i] times randn's."""
    d, n = 128, len(scores)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hkv, d, generator=g)
    along = q / (q * q).sum(-1, keepdim=True) * math.sqrt(d)  # a key of score 1
    m = n * L
    k = along[:, None] * torch.tensor(scores).repeat_interleave(L)[None, :, None, None]
    k = (k + 0.2 * torch.randn(B, m, Hkv, d, generator=g)).view(B * n, L, Hkv, d).transpose(1, 2)
    v = torch.randn(B * n, Hkv, L, d, generator=g)
    c = dict(q=q.to(torch.bfloat16).to(DEV), seq_lens=torch.full((B,), m, dtype=torch.int32, device=DEV),
             cu_q=torch.arange(B + 1, dtype=torch.int32, device=DEV),
             block_table=torch.arange(B * n, dtype=torch.int32, device=DEV).view(B, n))
    c["k_pages"], c["k_scale"] = (x.to(DEV) for x in R.quantise(k))
    c["v_pages"], s = R.quantise(v)
    s = s.view(B, n, Hkv, 1) * torch.tensor([2.0 ** x for x in spread]).view(1, n, 1, 1)
    c["v_pages"], c["v_scale"] = c["v_pages"].to(DEV), s.view(B * n, Hkv, 1).contiguous().to(DEV)
    return c


def check(c):
    """|error| <= half a step of the weights' type on every weight, 2^-8 of the output, and what the
    scores' errors make of the weights and their sum.  fp16 weights are held so that the largest of a
    row and tile is 2^4 at least: one below 2^-18 of it is off by 2^-29 of it at most, 64 of a tile by
    2^-23 of p v, with codes v <= 448 where the largest code of a token's 128 is above 64: below
    2^-20 of the largest sum p|v| of the row.
    Scores: the terms' absolute sum is below 80 (60 along the query, 16 and less of the rest), 128
    additions off by 2^-23 of it at most: 1.2e-3; a query's part below 2^-17 of its largest value
    may be lost: 2^-17 * 3.5 * 540 / 11.3 = 1.3e-3, with sum |k| = 60 * 0.088 * 128 * 0.8."""
    ro, rl, size = R.attend(c)
    score = 2.5e-3
    for kernel in KERNELS:  # (the definition takes longer than they do)
        out, lse = run(c, kernel)
        tol = (WEIGHT[kernel] + 2 * score) * size + 2.0 ** -8 * ro.abs() + 2.0 ** -20 * size.amax(-1, keepdim=True)
        worst = (out - ro).abs() / tol
        assert torch.isfinite(out).all(), kernel
        assert worst.max() <= 1.0, f"{kernel}: off by {worst.max():.3g} of the tolerance"
        assert (lse - rl).abs().max() <= score, kernel


@pytest.mark.parametrize("ratio", [0, 10, 20, 26, 40, 60])
def test_v_scales_far_apart(ratio):
    """Long runs, so that a warp takes several tiles of a sequence: V scales 2^ratio apart, falling
    or rising along it, against scores that rise or fall."""
    B, Hkv, n = 40, 12, 12  # 480 items of 12 tiles: some twenty tiles and more a CTA
    half = n // 2
    for seed, (scores, spread) in enumerate([
        ([-50.0] * half + [0.0] * half, [ratio] * half + [0] * half),     # large scales, then all the weight on small ones
        ([0.0] * half + [-50.0] * half, [0] * half + [ratio] * half),
        ([0.0] * half + [-30.0] * half, [0] * half + [ratio] * half),     # a weight of 2^-43 on the large scales
        ([-30.0] * half + [0.0] * half, [ratio] * half + [0] * half),
        ([0.0] * n, [ratio * (i % 2) for i in range(n)]),
        ([-60.0, 0.0, -20.0] * (n // 3), [2 * ratio // (i + 1) for i in range(n)]),
    ]):
        check(tiles_of_a_sequence(scores, spread, B, Hkv, seed))


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_row_keeps_its_bits_beside_others(kernel):
    """Rows of one row tile of which some see the end of a block with a scale 2^40 times the others'
    and the next do not: window 320 over 390 tokens, the first block left at row 383."""
    B, n, d, G, window = 20, 40, 128, 4, 320
    c = R.make_case([n] * B, [390] * B, 2 * G, 2, d, fp8=True, seed=3, device=DEV)
    c["v_scale"][c["block_table"][:, 0].long()] *= 2.0 ** 40
    out, lse = run(c, kernel, window=window)
    ro, rl, size = R.attend(c, window)
    tol = (WEIGHT[kernel] + 2.0 ** -11) * size + 2.0 ** -8 * ro.abs() + 2.0 ** -20 * size.amax(-1, keepdim=True)
    assert ((out - ro).abs() <= tol).all()
    assert (lse - rl).abs().max() <= 6.5e-4


@pytest.mark.parametrize("kernel", KERNELS)
def test_bits_of_the_weights(kernel):
    """Two tokens of opposite values and close weights: the output is the difference of the weights,
    so that the rounding of the weights shows beside the output's.  One-hot queries and keys: the
    scores are exact products, off by 2^-20 at most after the change of base."""
    B, d = 48, 128
    g = torch.Generator().manual_seed(7)
    c = R.make_case([2] * B, [2] * B, 2, 2, d, fp8=True, seed=7, device=DEV)
    q = torch.zeros(2 * B, 2, d)
    q[..., 77] = torch.rand(2 * B, 2, generator=g) + 0.5
    c["q"] = q.to(torch.bfloat16).to(DEV)
    k = torch.zeros(c["k_pages"].shape)
    k[:, :, :2, 77] = torch.randint(1, 120, (k.shape[0], 2, 2), generator=g).float()
    v = torch.zeros(k.shape)
    v[:, :, 0], v[:, :, 1] = 1.0, -1.0
    c["k_pages"], c["v_pages"] = k.to(R.E4M3).to(DEV), v.to(R.E4M3).to(DEV)
    c["k_scale"] = torch.full_like(c["k_scale"], 2.0 ** -10)
    c["v_scale"] = torch.full_like(c["v_scale"], 0.75)
    out, lse = run(c, kernel, softmax_scale=1.0)
    ro, rl, size = R.attend(c, scale=1.0)
    assert (ro[1::2].abs() < 0.1 * size[1::2]).all()  # (the second row of each sequence sees both)
    tol = (WEIGHT[kernel] + 2.0 ** -18) * size + 2.0 ** -8 * ro.abs()
    assert ((out - ro).abs() <= tol).all()
    assert (lse - rl).abs().max() <= 2.0 ** -20


# ------------------------------------------------------------------ queries


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_of_very_different_size(kernel):
    """A row 2^40 times another, a row of zeros and rows of ordinary size, in every place of a row
    tile: each is as exact as alone."""
    G, T = 4, 12
    for seed in range(4):
        c = R.make_case([T], [200], 2 * G, 2, 128, fp8=True, seed=30 + seed, device=DEV)
        big = (torch.arange(T)[:, None] * 8 + torch.arange(2 * G)) % 7 == seed
        zero = (torch.arange(T)[:, None] * 8 + torch.arange(2 * G)) % 11 == seed
        q = c["q"].cpu().float()
        q[big] *= 2.0 ** 40
        q[zero & ~big] = 0.0
        c["q"] = q.to(torch.bfloat16).to(DEV)
        out, lse = run(c, kernel)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        ro, rl, size = R.attend(c)
        tol = (WEIGHT[kernel] + 2.0 ** -11) * size + 2.0 ** -8 * ro.abs() + 2.0 ** -20 * size.amax(-1, keepdim=True)
        assert ((out - ro).abs() <= tol)[~big].all()
        # a query's part below 2^-17 of its largest value may be lost: 2^-17 max|q| sum |k| / sqrt(d),
        # below 2^-17 * 5 * 128 * 0.9 / 11.3 = 4e-4, beside 2.5e-4 of the sums
        assert (lse - rl).abs()[~big].max() <= 6.5e-4
        assert ((lse - rl).abs() <= 2.0 ** -16 * rl.abs() + 6.5e-4)[big].all()


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_query_that_is_no_number_spoils_its_own_row_only(kernel):
    """Infinities and NaN in some rows, beside rows of values above fp16's largest."""
    G, T = 4, 12
    c = R.make_case([T], [200], 2 * G, 2, 128, fp8=True, seed=40, device=DEV)
    q = c["q"].cpu().float() * 2.0 ** 17
    bad = (torch.arange(T)[:, None] * 8 + torch.arange(2 * G)) % 9 == 2
    q[..., 5][bad] = torch.tensor([math.inf, -math.inf, math.nan]).repeat(len(q))[: int(bad.sum())]
    c["q"] = q.to(torch.bfloat16).to(DEV)
    scale = 2.0 ** -17 / math.sqrt(128)
    out, lse = run(c, kernel, softmax_scale=scale)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    c["q"] = torch.where(bad[..., None], 0.0, c["q"].cpu().float()).to(torch.bfloat16).to(DEV)
    ro, rl, size = R.attend(c, scale=scale)
    tol = (WEIGHT[kernel] + 2.0 ** -11) * size + 2.0 ** -8 * ro.abs() + 2.0 ** -20 * size.amax(-1, keepdim=True)
    assert ((out - ro).abs() <= tol)[~bad].all()
    assert (lse - rl).abs()[~bad].max() <= 6.5e-4


@pytest.mark.parametrize("size", [1.0, 2.0 ** -100, 2.0 ** 126])
@pytest.mark.parametrize("kernel", KERNELS)
def test_small_values_of_a_query(kernel, size):
    """Row x has size at dim 0 and size 2^-x at dim 77, the only one where the keys are not zero: the
    lse of a row that sees one token is 2^-x k.  Exact from 2^-9 on, else off by 2^-17 at most.  (The
    size of the row does not count: the score scale takes it back.)"""
    T, d, G = 40, 128, 1
    q = torch.zeros(T, 1, d, dtype=torch.float64)
    q[:, 0, 0] = size
    q[:, 0, 77] = size * 2.0 ** -torch.arange(T, dtype=torch.float64)
    k = torch.zeros(1, 1, L, d)
    k[0, 0, :T, 77] = 96.0
    c = dict(q=q.to(torch.bfloat16).to(DEV), k_pages=k.to(R.E4M3).to(DEV), v_pages=torch.ones(1, 1, L, d).to(R.E4M3).to(DEV),
             k_scale=torch.ones(1, 1, 1, device=DEV), v_scale=torch.ones(1, 1, 1, device=DEV),
             block_table=torch.zeros(1, 1, dtype=torch.int32, device=DEV),
             seq_lens=torch.tensor([T], dtype=torch.int32, device=DEV), cu_q=torch.tensor([0, T], dtype=torch.int32, device=DEV))
    scale = 1.0 / size if size < 2.0 ** 120 else 2.0 ** -126
    _, lse = run(c, kernel, window=1, softmax_scale=scale)
    x = torch.arange(T, dtype=torch.float64)
    want = 96.0 * c["q"][:, 0, 77].cpu().double() * scale
    lost = torch.where(x <= 9, 0.0, 96.0 * 2.0 ** -17)
    assert ((lse[:, 0] - want).abs() <= lost + 2.0 ** -22 * want).all()
