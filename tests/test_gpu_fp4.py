"""4-bit pages: what qk_norm_rope_append writes, what attn_chunk_paged makes of them and what
kv_read_paged (all formats) gives back, against 64-bit definitions."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged
from tests import chunk_ref as R
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _append_case(q_lens, seq_lens, Hq, Hkv, block_len, rot, seed=0, gain=1.0, **kw):
    c = R.make_case(q_lens, seq_lens, Hq, Hkv, 128, block_len=block_len, seed=seed, device=DEV, **kw)
    g = c["gen"]
    T = c["q"].shape[0]
    c["qkv"] = (torch.randn(T, (Hq + 2 * Hkv) * 128, generator=g) * gain).bfloat16().to(DEV)
    c["cos"] = c["sin"] = None
    if rot:
        c["cos"], c["sin"] = paged.rotation_tables(c["block_table"].shape[1] * block_len, rot, device=DEV)
    n = c["k_pages"].shape[0]
    for x in "kv":  # what was there before
        c[x + "_pages"], c[x + "_scale"] = F.random_pages(n, Hkv, block_len, 128, g, DEV)
    return c


def _check_block(y, codes, scales, head):
    """y [.., d] in 64 bits and its codes' values and scales.  y is off by 2^-19 of itself at most (fp32 norm
    and rotation; the two summands of a rotation may cancel: relative to the head's largest), so the scale is
    the nearest e4m3 to a value that near, and every code the nearest to one."""
    b = y.unflatten(-1, (-1, 16))
    slack = 2.0 ** -19 * y.abs().amax(-1)[..., None]
    t = (b.abs().amax(-1) / (6 * head)).clamp_max(448.0)
    # half an e4m3 step: 2^-4 of the power of two below, 2^-10 at least
    half = torch.maximum(2.0 ** (torch.floor(torch.log2(t.clamp_min(2.0 ** -6))) - 4), torch.tensor(2.0 ** -10).double())
    assert ((scales - t).abs() <= half * (1 + 2.0 ** -18) + slack / (6 * head)).all()
    by = (scales * head)[..., None]
    x = torch.where(by > 0, b / by, 0.0)
    off = (x.clamp(-6, 6) - codes.unflatten(-1, (-1, 16))).abs()
    best = (x.clamp(-6, 6)[..., None] - F.VALUES).abs().amin(-1)
    ok = off <= best + torch.where(by > 0, 2 * slack[..., None] / by, 0.0) + 2.0 ** -20 * x.abs()
    assert ok.all(), (~ok).sum()


@pytest.mark.parametrize("q_lens,seq_lens,Hq,Hkv,block_len,rot,paired,per_head", [
    ((1,), (1,), 4, 1, 64, 128, False, False),
    ((1, 1, 1), (64, 65, 200), 8, 2, 64, 128, True, False),
    ((70, 0, 3, 1), (70, 5, 300, 129), 12, 4, 128, 64, False, True),
    ((33, 9), (100, 9), 5, 5, 320, 16, False, True),
    ((33, 9), (100, 9), 10, 2, 64, 16, True, False),
    ((40,), (47,), 2, 1, 64, 48, False, False),
    ((40,), (47,), 34, 17, 64, 0, False, False),
    ((257, 300), (300, 300), 16, 8, 64, 112, False, False),
])
def test_append(q_lens, seq_lens, Hq, Hkv, block_len, rot, paired, per_head):
    c = _append_case(q_lens, seq_lens, Hq, Hkv, block_len, rot, spare_rows=2)
    g = torch.Generator().manual_seed(5)
    qw, kw = ((1 + 0.2 * torch.randn(h, 128, generator=g)).bfloat16().to(DEV) for h in (Hq, Hkv))
    if not per_head:
        qw, kw = qw[0].contiguous(), kw[0].contiguous()
    heads = [(0.25 + 2 * torch.rand(Hkv, generator=g)).to(DEV), None]
    before = {x: (c[x + "_pages"].clone(), c[x + "_scale"].clone()) for x in "kv"}
    q, k, v = paged.split_qkv(c["qkv"], Hq, Hkv)
    q_out = skv.qk_norm_rope_append(q, k, v, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    cos=c["cos"], sin=c["sin"], q_weight=qw, k_weight=kw, interleaved=paired,
                                    k_scale=c["k_scale"], v_scale=c["v_scale"], k_head_scale=heads[0], v_head_scale=heads[1])
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    where = R.places(c)
    rows = torch.tensor([r for _, _, r in where])
    pos = torch.tensor([p for _, p, _ in where])
    page = torch.tensor([int(c["block_table"][b, p // block_len]) for b, p, _ in where])
    at = pos % block_len
    yq = R.norm_rope(q[rows.to(DEV)], qw, c["cos"], c["sin"], pos, 1e-6, paired)
    assert ((q_out.cpu().double()[rows] - yq).abs() <= 2.0 ** -8 * yq.abs() + 2.0 ** -18 * yq.abs().amax(-1, keepdim=True)).all()
    ys = {"k": R.norm_rope(k[rows.to(DEV)], kw, c["cos"], c["sin"], pos, 1e-6, paired), "v": v[rows.to(DEV)].cpu().double()}
    for x, h in zip("kv", heads):
        codes, scales = F.values_of(c[x + "_pages"])[page, :, at], F.scales_of(c[x + "_scale"])[page, :, at]
        h64 = torch.ones(Hkv, 1).double() if h is None else h.cpu().double()[:, None]
        _check_block(ys[x], codes, scales, h64)
        # nothing else changed
        for new, old in zip((c[x + "_pages"], c[x + "_scale"]), before[x]):
            new, old = new.view(torch.uint8).cpu().clone(), old.view(torch.uint8).cpu()
            new[page, :, at] = old[page, :, at]
            assert torch.equal(new, old)


def test_append_values_are_exact_quantisations():
    """Values without norm and rotation are what the formula gives, bit for bit: magnitudes of many
    sizes, blocks of zeros, ties between two codes, infinities, NaN."""
    Hkv, T = 2, 64
    c = _append_case((T,), (T,), 2, Hkv, 64, 0)
    g = torch.Generator().manual_seed(8)
    v = torch.randn(T, Hkv, 8, 16, generator=g) * torch.exp2(torch.randint(-14, 12, (T, Hkv, 8, 1), generator=g).float())
    v[0, 0, 0] = 0
    v[1, 0, 0] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6.0])
    v[2, 0, 0, 3] = math.inf
    v[3, 0, 0, 5] = math.nan
    v[4, 1, 7] = 3e38
    v = v.flatten(2).bfloat16().to(DEV)
    q = torch.zeros(T, 2, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(T, Hkv, 128, dtype=torch.bfloat16, device=DEV)
    head = torch.tensor([1.0, 0.3], device=DEV)
    skv.qk_norm_rope_append(q, k, v, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                            k_scale=c["k_scale"], v_scale=c["v_scale"], v_head_scale=head)
    page = int(c["block_table"][0, 0])
    got = F.values_of(c["v_pages"])[page].transpose(0, 1).unflatten(-1, (-1, 16))
    scales = F.scales_of(c["v_scale"])[page].transpose(0, 1)
    y = v.cpu().float().unflatten(-1, (-1, 16))
    h = head.cpu()[:, None]
    want = (y.abs().amax(-1) / (6 * h)).clamp_max(448.0).to(torch.float8_e4m3fn).double()
    assert math.isnan(scales[3, 0, 0]) and math.isnan(want[3, 0, 0])
    ok = ~torch.isnan(want)
    assert torch.equal(scales[ok], want[ok])
    x = y / (want.float() * h)[..., None]
    x = torch.where((want > 0)[..., None], x, 0.0).double().clamp(-6, 6)
    step = (x[..., None].abs() - F.E2M1).abs()
    near = step == step.amin(-1, keepdim=True)
    even = near & (torch.arange(8) % 2 == 0)
    code = torch.where(near.sum(-1) > 1, even.int().argmax(-1), near.int().argmax(-1))
    val = torch.copysign(F.E2M1[code], x)
    assert torch.equal(got[ok], val[ok])
    assert (F.values_of(c["k_pages"])[page] * F.scales_of(c["k_scale"])[page].repeat_interleave(16, -1) == 0).all()


def test_append_bad_head_scales_and_places():
    """A head scale that is no usable number stores zeros; tokens without a page are dropped."""
    Hkv = 4
    c = _append_case((5,), (70,), 4, Hkv, 64, 0)
    c["block_table"][0, 1] = -1  # tokens 65 .. 69 lie there
    q, k, v = paged.split_qkv(c["qkv"], 4, Hkv)
    head = torch.tensor([1.0, 0.0, math.nan, 1e30], device=DEV)
    before = c["k_pages"].clone()
    args = (c["seq_lens"], c["cu_q"], c["block_table"])
    kw = dict(k_scale=c["k_scale"], v_scale=c["v_scale"], k_head_scale=head, v_head_scale=-head)
    skv.qk_norm_rope_append(q, k, v, c["k_pages"], c["v_pages"], *args, **kw)
    assert torch.equal(before, c["k_pages"])
    c["block_table"][0, 1] = 1
    skv.qk_norm_rope_append(q, k, v, c["k_pages"], c["v_pages"], *args, **kw)
    ks, vs = F.scales_of(c["k_scale"])[1, :, 1:6], F.scales_of(c["v_scale"])[1, :, 1:6]
    assert (ks[0] > 0).all() and (ks[1:] == 0).all() and (vs == 0).all()
    k16, v16 = skv.kv_read_paged(c["k_pages"], c["v_pages"], torch.tensor([0, 5], dtype=torch.int32, device=DEV),
                                 c["block_table"], n_tokens=5, starts=torch.tensor([65], dtype=torch.int32, device=DEV), **kw)
    assert (k16[:, 1:] == 0).all() and (v16 == 0).all() and (k16[:, 0] != 0).any()


# ------------------------------------------------------------------ attention

ATTN = [
    # q_lens, seq_lens, Hq, Hkv, block_len, max_q_len
    ((1,), (1,), 1, 1, 64, 1),
    ((1,), (5,), 16, 1, 64, 1),
    ((1, 1, 1, 0), (64, 65, 1000, 7), 8, 2, 64, 1),
    ((1, 1), (4000, 130), 64, 8, 128, 1),
    ((3, 1, 2), (300, 64, 129), 10, 2, 320, 3),
    ((5, 5), (700, 5), 40, 8, 64, 5),
    ((2, 2, 2), (900, 65, 64), 32, 2, 64, 2),
    ((40, 1, 7), (40, 333, 500), 8, 2, 64, None),
    ((129,), (129,), 12, 4, 64, None),
    ((300, 17), (1500, 17), 16, 2, 128, None),
    ((6,), (200,), 136, 1, 64, None),
]


@pytest.mark.parametrize("q_lens,seq_lens,Hq,Hkv,block_len,max_q_len", ATTN)
def test_attention(q_lens, seq_lens, Hq, Hkv, block_len, max_q_len):
    c = F.make_case("fp4", q_lens, seq_lens, Hq, Hkv, 128, block_len=block_len, seed=3, device=DEV)
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, **F.pages_of(c))
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    R.check_attention(c["dense"], out, lse)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (64, 4), (100, 70), (500, 1)])
@pytest.mark.parametrize("max_q_len", [8, None])
def test_attention_window(window, n_sink, max_q_len):
    q_lens, seq_lens = (8, 1, 5), (900, 70, 333)
    c = F.make_case("fp4", q_lens, seq_lens, 8, 2, 128, seed=4, device=DEV)
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, window=window, n_sink=n_sink, **F.pages_of(c))
    R.check_attention(c["dense"], out, lse, window=window, n_sink=n_sink)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (2, 1), (64, 4), (100, 70), (500, 1)])
@pytest.mark.parametrize("Hq,Hkv,q_lens", [(8, 2, (2, 1, 2)), (8, 1, (1, 1, 1)), (3, 3, (8, 1, 7)), (6, 2, (2, 2, 0))])
def test_attention_window_few_rows(window, n_sink, Hq, Hkv, q_lens):
    """Up to 8 rows of a KV head."""
    c = F.make_case("fp4", q_lens, (900, 70, 333), Hq, Hkv, 128, seed=14, device=DEV)
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max(q_lens), window=window, n_sink=n_sink, **F.pages_of(c))
    assert skv.device_error() == 0
    R.check_attention(c["dense"], out, lse, window=window, n_sink=n_sink)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (8, 8), (64, 8)])
def test_attention_few_rows_many_sequences(Hq, Hkv):
    """More items than CTAs, some of them empty or of one token: runs that begin and end inside items."""
    lens = [1 + (i * 977) % 1500 for i in range(60)] + [0, 1, 64]
    q_lens = [1] * 60 + [0, 1, 1]
    c = F.make_case("fp4", q_lens, lens, Hq, Hkv, 128, seed=18, device=DEV)
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=1, **F.pages_of(c))
    R.check_attention(c["dense"], out, lse)


@pytest.mark.parametrize("max_q_len", [2, 3, 12, None])
def test_attention_unseen_and_missing_pages(max_q_len):
    """NaN scales behind the last token and in pages of nobody change nothing; entries outside the cache
    read as zeros."""
    c = F.make_case("fp4", (3, 1), (200, 100), 8, 2, 128, seed=6, device=DEV)
    c["block_table"][0, 1] = 1 << 20
    for x in "kv":
        s = c[x + "_scale"].view(torch.uint8)
        for b, m in enumerate((200, 100)):
            s[int(c["block_table"][b, (m - 1) // 64]), :, m % 64:] = 0x7F
        used = c["block_table"][c["block_table"] >= 0].tolist()
        for p in set(range(s.shape[0])) - set(used):
            s[p] = 0xFF
    F.with_dense(c)
    dense = {x: torch.nan_to_num(c["dense"][x]) if x.endswith("pages") else c["dense"][x] for x in c["dense"]}
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, **F.pages_of(c))
    R.check_attention(dense, out, lse)


@pytest.mark.parametrize("max_q_len", [1, 2, None])
def test_attention_far_scales(max_q_len):
    """Queries, head scales and block scales far from 1: largest blocks of one token 2^17 times another's,
    head scales of 2^30 and 2^-30; scores stay below 2^5."""
    c = F.make_case("fp4", (1, 1), (150, 400), 16, 2, 128, seed=7, device=DEV)
    c["k_head_scale"] = torch.tensor([2.0 ** 30, 2.0 ** -30], device=DEV)
    c["v_head_scale"] = torch.tensor([2.0 ** -40, 2.0 ** 40], device=DEV)
    q = c["q"].float()
    q[:, :8] *= 2.0 ** -30
    q[:, 8:] *= 2.0 ** 30
    c["q"] = q.bfloat16()
    g = torch.Generator().manual_seed(1)
    by = torch.exp2(torch.randint(-8, 9, c["v_scale"].shape[:3], generator=g).float())[..., None]
    c["v_scale"] = (c["v_scale"].float().cpu() * by).to(torch.float8_e4m3fn).to(DEV)
    F.with_dense(c)
    c["dense"]["q"] = c["q"]
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, **F.pages_of(c))
    R.check_attention(c["dense"], out, lse)


def test_attention_flat_after_a_spike():
    """One token that outweighs each of the others by 2^20, and 50000 of those: together they count."""
    n = 50000
    c = F.make_case("fp4", (1,), (n,), 4, 1, 128, seed=2, device=DEV)
    L = 64
    q = torch.zeros(1, 4, 128)
    q[..., 0] = 8.0
    c["q"] = q.bfloat16().to(DEV)
    c["k_pages"].zero_()
    c["k_scale"] = torch.full_like(c["k_scale"].view(torch.uint8), 0x38).view(torch.float8_e4m3fn)  # 1.0
    c["k_head_scale"] = c["v_head_scale"] = None
    first = int(c["block_table"][0, 0])
    c["k_pages"][first, 0, 3, 0] = 7  # 6.0
    scale = 20 * math.log(2) / 48  # s = 20 ln 2 for that token, 0 for the others
    F.with_dense(c)
    c["dense"]["q"] = c["q"]
    for max_q_len in (1, None):
        out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                        max_q_len=max_q_len, softmax_scale=scale, **F.pages_of(c))
        R.check_attention(c["dense"], out, lse, scale=scale)


@pytest.mark.parametrize("max_q_len", [1, 2, None])
@pytest.mark.parametrize("step", [0.02, 0.5])
def test_attention_scores_that_rise(max_q_len, step):
    """Scores that grow from token to token, slowly or by more than fp16's range within a tile: the maximum
    moves in every tile."""
    n = 700
    c = F.make_case("fp4", (1, 1), (n, 300), 8, 2, 128, seed=15, device=DEV)
    q = torch.zeros(2, 8, 128)
    q[..., 0] = 1.0
    q[..., 16] = 1.0
    c["q"] = q.bfloat16().to(DEV)
    # dim 0: code 1.0 times a scale, so that the score is the token's scale: the nearest e4m3 of step * t
    c["k_pages"].zero_()
    c["k_pages"][..., 0] = 2
    s = torch.zeros(c["k_scale"].shape)
    for b, m in enumerate((n, 300)):
        t = torch.arange(m)
        s[c["block_table"][b].cpu().long()[t // 64], :, t % 64, 0] = (step * t)[:, None].float()
    c["k_scale"] = s.to(torch.float8_e4m3fn).to(DEV)
    c["k_head_scale"] = None
    F.with_dense(c)
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, softmax_scale=1.0, **F.pages_of(c))
    ro, rl, size = R.attend(c["dense"], scale=1.0)
    # scores up to 448 in base 2 up to 2^10: each off by 2^-23 of that at most, and so a weight by 2^-13
    assert ((lse.cpu().double() - rl).abs() <= 2.0 ** -22 * rl.abs() + 2.5e-4).all()
    assert ((out.cpu().double() - ro).abs() <= 2.0 ** -8 * (ro.abs() + size) + 2.0 ** -11 * size).all()


@pytest.mark.parametrize("max_q_len", [1, 2, None])
@pytest.mark.parametrize("gain", [2.0 ** 18, 2.0 ** 24, 2.0 ** 27])
@pytest.mark.parametrize("Hq", [8, 32])
@pytest.mark.parametrize("n", [64, 900])
def test_attention_huge_scores(n, gain, max_q_len, Hq):
    """Scores up to 6 * 2^27 (base 2: past 2^29, where neighbouring numbers are 64 apart): tokens with the largest
    score share the weight, and nothing overflows.  Rows of several items are joined by their lse, which 32 bits
    hold to 2^-24 of itself: there (n = 900) a weight is off by 2^-22 |lse| of itself, and where that is more than
    all of it the output is still a mean of the rows that share the largest score."""
    c = F.make_case("fp4", (1, 1), (n, min(n, 300)), Hq, 2, 128, seed=19, device=DEV)
    q = torch.zeros(2, Hq, 128)
    q[..., 0] = 1.0
    c["q"] = q.bfloat16().to(DEV)
    g = torch.Generator().manual_seed(3)
    c["k_pages"].zero_()
    c["k_pages"][..., 0] = torch.randint(0, 8, c["k_pages"].shape[:3], generator=g, dtype=torch.uint8).to(DEV)
    c["k_scale"] = torch.full_like(c["k_scale"].view(torch.uint8), 0x38).view(torch.float8_e4m3fn)  # 1.0
    c["k_head_scale"] = None
    F.with_dense(c)
    c["dense"]["q"] = c["q"]
    out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                    max_q_len=max_q_len, softmax_scale=gain, **F.pages_of(c))
    ro, rl, size = R.attend(c["dense"], scale=gain)
    # equal scores are equal in 32 bits too; others lie 2^17 and more lower
    out, lse = out.cpu().double(), lse.cpu().double()
    assert ((lse - rl).abs() <= 2.0 ** -21 * rl.abs()).all()
    tol = 2.0 ** -8 * (ro.abs() + size) + 2.0 ** -12 * size
    if n > 64:
        most = c["dense"]["v_pages"].abs().amax()
        tol += torch.clamp(2.0 ** -22 * rl.abs()[..., None] * size, max=2 * most)
    assert torch.isfinite(out).all() and ((out - ro).abs() <= tol).all()


@pytest.mark.parametrize("n", [1, 5, 20])
def test_attention_cut_in_chunks(n):
    """Few rows over many tokens: on the tensor cores every row's tokens are dealt to several items."""
    c = F.make_case("fp4", (n, 3), (20000, 9000), 16, 2, 128, block_len=128, seed=16, device=DEV)
    for max_q_len in (n, None):
        out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                        max_q_len=max(max_q_len, 3) if max_q_len else None, **F.pages_of(c))
        R.check_attention(c["dense"], out, lse)


def test_queries_with_infinities_spoil_their_rows_only():
    c = F.make_case("fp4", (4,), (300,), 8, 2, 128, seed=17, device=DEV)
    want, _ = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"], **F.pages_of(c))
    c["q"][1, 3, 7] = math.inf
    c["q"][2, 0, 100] = math.nan
    for max_q_len in (4, None):
        out, lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                        max_q_len=max_q_len, **F.pages_of(c))
        bad = torch.zeros(4, 8, dtype=torch.bool, device=DEV)
        bad[1, 3] = bad[2, 0] = True
        assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(lse), bad)
        assert ((out.float() - want.float())[~bad].abs() <= 2.0 ** -7 * want.float()[~bad].abs() + 2.0 ** -7).all()


def test_strided_pages_and_float4_dtype():
    """Pages as every other token row, page and head of a larger buffer; codes as float4_e2m1fn_x2."""
    c = F.make_case("fp4", (1, 2), (300, 130), 8, 2, 128, seed=11, device=DEV)
    n, Hkv, L, w = c["k_pages"].shape
    for x in "kv":
        big = torch.full((n, 2, Hkv, L, 2, w), 0x77, dtype=torch.uint8, device=DEV)
        view = big[:, 0, :, :, 1]
        view.copy_(c[x + "_pages"])
        c[x + "_pages"] = view
    want = skv.attn_chunk_paged(c["q"], c["k_pages"].contiguous(), c["v_pages"].contiguous(), c["seq_lens"], c["cu_q"],
                                c["block_table"], max_q_len=2, **F.pages_of(c))
    kinds = [torch.uint8] + ([torch.float4_e2m1fn_x2] if hasattr(torch, "float4_e2m1fn_x2") else [])
    for kind in kinds:
        k, v = c["k_pages"].view(kind), c["v_pages"].view(kind)
        out, lse = skv.attn_chunk_paged(c["q"], k, v, c["seq_lens"], c["cu_q"], c["block_table"], max_q_len=2, **F.pages_of(c))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    R.check_attention(c["dense"], out, lse)
    k16, v16 = skv.kv_read_paged(c["k_pages"], c["v_pages"], c["cu_q"], c["block_table"], n_tokens=3, **F.pages_of(c))
    assert torch.equal(k16[0].cpu(), c["dense"]["k_pages"][int(c["block_table"][0, 0]), :, 0].bfloat16())


# ------------------------------------------------------------------ reading back


@pytest.mark.parametrize("fmt,d", [("bf16", 64), ("bf16", 128), ("fp8", 128), ("fp4", 128)])
@pytest.mark.parametrize("lens,starts,Hkv,block_len", [
    ((1,), None, 1, 64),
    ((70, 0, 1, 200), (0, 3, 64, 100), 2, 64),
    ((129, 31), (1, 63), 3, 192),
    ((33, 1000), None, 8, 64),
])
def test_read(fmt, d, lens, starts, Hkv, block_len):
    seq = [n + (starts[i] if starts else 0) for i, n in enumerate(lens)]
    c = F.make_case(fmt, lens, [max(1, s) for s in seq], Hkv, Hkv, d, block_len=block_len, seed=12, device=DEV)
    T = sum(lens)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    outs = [torch.full((T + 3, Hkv, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k, v = skv.kv_read_paged(c["k_pages"], c["v_pages"], c["cu_q"], c["block_table"], starts=st, k_out=outs[0],
                             v_out=outs[1], **F.pages_of(c))
    for x, got in (("k", k), ("v", v)):
        full = c["dense"][x + "_pages"] if fmt == "fp4" else R.dense(c[x + "_pages"], c[x + "_scale"])
        rows = []
        for b, n in enumerate(lens):
            t = torch.arange(n) + (starts[b] if starts else 0)
            rows.append(full[c["block_table"][b].cpu().long()[t // block_len], :, t % block_len])
        want = torch.cat(rows)
        # one fp32 product (4-bit: two) and one rounding to bf16
        assert ((got[:T].cpu().double() - want).abs() <= (2.0 ** -9 + 2.0 ** -22) * 2 * want.abs()).all()
        if fmt == "bf16":
            assert torch.equal(got[:T].cpu().double(), want)
        assert (got[T:] == 7).all()


def test_read_bad_places_and_strides():
    c = F.make_case("fp4", (4, 4), (100, 100), 2, 2, 128, seed=13, device=DEV)
    c["block_table"][0, 0] = -3
    starts = torch.tensor([62, 126], dtype=torch.int32, device=DEV)  # the second runs past the table
    head_major = [torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k, v = skv.kv_read_paged(c["k_pages"], c["v_pages"], c["cu_q"], c["block_table"], starts=starts,
                             k_out=head_major[0].transpose(0, 1), v_out=head_major[1].transpose(0, 1), **F.pages_of(c))
    assert (head_major[0][:, :2] == 0).all() and (head_major[0][:, 6:] == 0).all()
    page = int(c["block_table"][0, 1])
    assert torch.equal(head_major[0][:, 2].cpu(), c["dense"]["k_pages"][page, :, 0].bfloat16())
    assert torch.equal(head_major[1][:, 3].cpu(), c["dense"]["v_pages"][page, :, 1].bfloat16())
    starts[0] = -1
    k, _ = skv.kv_read_paged(c["k_pages"], c["v_pages"], c["cu_q"], c["block_table"], n_tokens=8, starts=starts, **F.pages_of(c))
    assert (k[0] == 0).all()


# ------------------------------------------------------------------ together


def test_step_over_4bit_pages_captured_and_replayed():
    """chunk_step (append, then attention over what was written) in a graph, replayed with other lengths:
    the result is the attention over the pages as kv_read_paged gives them."""
    Hq, Hkv, B, L = 16, 2, 3, 64
    g = torch.Generator().manual_seed(21)
    pages = paged.fp4_pages(12, Hkv, L, device=DEV)
    k_pages, v_pages, k_scale, v_scale = pages
    table = torch.randperm(12, generator=g)[:B * 4].view(B, 4).int().to(DEV)
    cos, sin = paged.rotation_tables(4 * L, 128, device=DEV)
    w = torch.ones(128, device=DEV)
    T = 40
    qkv = torch.empty(T, (Hq + 2 * Hkv) * 128, dtype=torch.bfloat16, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)

    def step():
        return paged.chunk_step(qkv, Hq, Hkv, k_pages, v_pages, lens, cu, table, cos=cos, sin=sin, q_weight=w, k_weight=w,
                                k_scale=k_scale, v_scale=v_scale)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    have = [0] * B
    for n in ((20, 11, 9), (1, 0, 30), (7, 7, 7), (1, 1, 1)):
        have = [a + b for a, b in zip(have, n)]
        qkv.copy_(torch.randn(qkv.shape, generator=g).bfloat16())
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        cu.copy_(torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert skv.device_error() == 0
        c = dict(k_pages=F.dense(k_pages, k_scale, None), v_pages=F.dense(v_pages, v_scale, None), k_scale=None, v_scale=None,
                 seq_lens=lens, cu_q=cu, block_table=table)
        q = skv.qk_norm_rope_append(*paged.split_qkv(qkv, Hq, Hkv), k_pages, v_pages, lens, cu, table, cos=cos, sin=sin,
                                    q_weight=w, k_weight=w, k_scale=k_scale, v_scale=v_scale)
        R.check_attention(dict(c, q=q), out, lse)
