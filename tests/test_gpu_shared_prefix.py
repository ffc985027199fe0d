"""attn_shared_prefix_paged against the 64-bit definition of attention over each sequence's own pages."""

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged
from tests import chunk_ref as R
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def shared_case(fmt, d, groups, Hq, Hkv, block_len=64, seed=0, outside=(), **kw):
    """groups: [(prefix, [(new tokens, tokens behind the prefix with them), ..]), ..]; outside: the lengths of
    sequences of no group, which come last."""
    q_lens, seq_lens, cu = [], [], [0]
    for prefix, members in groups:
        for n, own in members:
            q_lens.append(n)
            seq_lens.append(prefix + own)
        cu.append(len(q_lens))
    for n, m in outside:
        q_lens.append(n)
        seq_lens.append(m)
    c = F.make_case(fmt, q_lens, seq_lens, Hq, Hkv, d, block_len=block_len, seed=seed, device=DEV, **kw)
    for j, (prefix, _) in enumerate(groups):
        if cu[j + 1] > cu[j]:
            blocks = prefix // block_len
            c["block_table"][cu[j]:cu[j + 1], :blocks] = c["block_table"][cu[j], :blocks].clone()
    c["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    c["prefix_lens"] = torch.tensor([p for p, _ in groups], dtype=torch.int32, device=DEV)
    c["dense"]["block_table"] = c["block_table"]
    return c


def run(c, **kw):
    out, lse = skv.attn_shared_prefix_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                            c["cu_groups"], c["prefix_lens"], **F.pages_of(c), **kw)
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    return out, lse


FORMATS = [("bf16", 64), ("bf16", 128), ("fp8", 128), ("fp4", 128)]
DECODE = [(1, 1), (1, 64), (1, 65), (1, 300), (1, 2)]
CASES = {
    "one token each": ([(640, DECODE)], 16, 2),
    "one sequence": ([(128, [(1, 1)])], 4, 1),
    "many rows": ([(2000 // 64 * 64, [(1, 10 + i) for i in range(40)])], 16, 2),
    "drafts": ([(320, [(5, 5), (3, 70), (5, 200)])], 10, 2),
    "ragged chunks": ([(704, [(70, 70), (1, 30), (131, 140)])], 8, 4),
    "groups": ([(64, [(1, 1), (1, 2)]), (0, [(2, 5)]), (1280, []), (192, [(1, 90), (0, 7), (4, 4)])], 12, 4),
    "outside": ([(256, [(1, 9), (1, 10)])], 8, 2),
    "wide group of heads": ([(192, [(1, 3), (1, 4), (1, 5)])], 136, 1),
}


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("small", [True, False])
def test_shared(fmt, d, name, small):
    groups, Hq, Hkv = CASES[name]
    outside = [(1, 77), (3, 3)] if name == "outside" else ()
    c = shared_case(fmt, d, groups, Hq, Hkv, seed=1, outside=outside, spare_rows=2)
    n = [m[0] for _, ms in groups for m in ms] + [m[0] for m in outside]
    most = max(sum(m[0] for m in ms) for _, ms in groups)
    kw = dict(max_q_len=max(n), max_group_rows=most) if small else {}
    out0 = torch.full_like(c["q"], 5.0)
    lse0 = torch.full(c["q"].shape[:2], 5.0, device=DEV)
    out, lse = run(c, out=out0, lse=lse0, **kw)
    R.check_attention(c["dense"], out, lse)
    assert (out[-2:] == 5).all() and (lse[-2:] == 5).all()


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 200, 10 ** 9, -5])
def test_prefix_lengths(fmt, d, prefix):
    """A prefix is cut to whole tiles that every new token sees: sequences that are really the same up to 256
    tokens, said to share any number."""
    c = shared_case(fmt, d, [(256, [(1, 1), (7, 8), (1, 40)])], 8, 2, seed=2)
    if prefix > 256:  # all of every table row then
        c["block_table"][:] = c["block_table"][2].clone()
        c["seq_lens"][:] = torch.tensor([257, 264, 296], dtype=torch.int32)
    c["prefix_lens"].fill_(prefix)
    out, lse = run(c, max_q_len=7)
    R.check_attention(c["dense"], out, lse)


@pytest.mark.parametrize("block_len", [64, 128, 320])
def test_long_prefix_is_cut_in_chunks(block_len):
    P = 9600
    for fmt, d in FORMATS:
        c = shared_case(fmt, d, [(P, [(1, 5), (1, 70), (2, 2)])], 16, 2, block_len=block_len, seed=3)
        for kw in (dict(max_q_len=2, max_group_rows=4), dict()):
            out, lse = run(c, **kw)
            R.check_attention(c["dense"], out, lse)


def test_broken_groups_read_and_write_in_bounds():
    """cu_groups that leave [0, B] or cover no sequence: clipped; the result is attn_chunk_paged's."""
    c = shared_case("bf16", 128, [(256, [(1, 1), (2, 8), (1, 40)])], 8, 2, seed=4)
    for cu in ([-3, 99], [2, 2], [3, 3], [5, 9], [1, 3]):
        c["cu_groups"].copy_(torch.tensor(cu, dtype=torch.int32))
        out, lse = run(c, max_q_len=2)
        R.check_attention(c["dense"], out, lse)


def test_sequence_without_new_tokens_may_have_given_its_pages_back():
    c = shared_case("bf16", 128, [(256, [(0, 1), (1, 8), (1, 40)])], 8, 2, seed=5)
    c["block_table"][0] = -1
    c["seq_lens"][0] = 0
    out, lse = run(c, max_q_len=1)
    R.check_attention(c["dense"], out, lse)


def test_scores_far_apart():
    """The prefix outweighs the rest, or the other way round, by all that fp32 can tell; tokens whose scores
    are -inf make no weight."""
    c = shared_case("bf16", 128, [(128, [(1, 64), (1, 3)])], 8, 2, seed=6)
    q = torch.zeros_like(c["q"])
    q[:, :4, 0] = 100.0
    q[:, 4:, 0] = -100.0
    c["q"] = c["dense"]["q"] = q
    first = c["block_table"][0, :2].long()
    for p, x in ((c["k_pages"], 50.0), (c["v_pages"], 3.0)):
        p[first, ..., 0] = x
    out, lse = run(c, max_q_len=1)
    ro, rl, size = R.attend(c["dense"])
    # scores up to 450: fp32 sums of one product each, base-2 arithmetic of numbers up to 2^10
    assert ((lse.cpu().double() - rl).abs() <= 2.0 ** -21 * rl.abs() + 2.5e-4).all()
    assert ((out.cpu().double() - ro).abs() <= 2.0 ** -8 * (ro.abs() + size) + 2.0 ** -11 * size).all()


def test_nan_in_the_prefix_reaches_its_rows_only():
    c = shared_case("bf16", 64, [(128, [(1, 5), (1, 9)]), (64, [(1, 5)])], 4, 2, seed=7)
    c["k_pages"][int(c["block_table"][0, 1]), 1, 5] = float("nan")
    out, lse = run(c, max_q_len=1)
    want, _ = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"], max_q_len=1)
    bad = torch.isnan(want)
    assert bad[:2, 2:].all() and not bad[:2, :2].any() and not bad[2].any()
    assert torch.equal(torch.isnan(out), bad)


def test_two_streams_and_graphs_at_once():
    """Two captured steps replayed on two streams at once, then with other lengths and groups."""
    cases = [shared_case(f, 128, [(640, DECODE), (64, [(2, 7)])], 16, 2, seed=s) for f, s in (("bf16", 8), ("fp4", 9))]
    graphs, outs = [], []
    for c in cases:
        run(c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(skv.attn_shared_prefix_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"],
                                                     c["block_table"], c["cu_groups"], c["prefix_lens"], **F.pages_of(c)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(3):
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert skv.device_error() == 0
        for c, (out, lse) in zip(cases, outs):
            R.check_attention(c["dense"], out, lse)
            if turn == 0:
                c["seq_lens"] -= torch.tensor([0, 3, 1, 100, 0, 1], dtype=torch.int32, device=DEV)
            if turn == 1:
                c["prefix_lens"].copy_(torch.tensor([320, 0], dtype=torch.int32))


def test_step_with_a_shared_prefix():
    """chunk_step with groups: the prompt first, then samples of it, over pages that the first step wrote."""
    Hq, Hkv, L, P = 16, 4, 64, 256
    g = torch.Generator().manual_seed(31)
    for fp4 in (False, True):
        if fp4:
            k_pages, v_pages, k_scale, v_scale = paged.fp4_pages(9, Hkv, L, device=DEV)
        else:
            k_pages, v_pages = (torch.zeros(9, Hkv, L, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            k_scale = v_scale = None
        cos, sin = paged.rotation_tables(P + L, 128, device=DEV)
        w = torch.ones(128, device=DEV)
        kw = dict(cos=cos, sin=sin, q_weight=w, k_weight=w, k_scale=k_scale, v_scale=v_scale)

        def ints(*x):
            return torch.tensor(x, dtype=torch.int32, device=DEV)

        def projection(T):
            return torch.randn(T, (Hq + 2 * Hkv) * 128, generator=g).bfloat16().to(DEV)

        paged.chunk_step(projection(P), Hq, Hkv, k_pages, v_pages, ints(P), ints(0, P), ints(3, 1, 7, 0)[None], **kw)
        table = torch.cat((ints(3, 1, 7, 0).expand(4, 4), ints(2, 4, 5, 8)[:, None]), 1).contiguous()
        qkv = projection(4)
        out, lse = paged.chunk_step(qkv, Hq, Hkv, k_pages, v_pages, ints(*[P + 1] * 4), ints(0, 1, 2, 3, 4), table,
                                    max_q_len=1, cu_groups=ints(0, 4), prefix_lens=ints(P), max_group_rows=4, **kw)
        q = skv.qk_norm_rope_append(*paged.split_qkv(qkv, Hq, Hkv), k_pages, v_pages, ints(*[P + 1] * 4), ints(0, 1, 2, 3, 4),
                                    table, **kw)
        c = dict(q=q, k_pages=k_pages, v_pages=v_pages, k_scale=None, v_scale=None, seq_lens=ints(*[P + 1] * 4),
                 cu_q=ints(0, 1, 2, 3, 4), block_table=table)
        if fp4:
            c.update(k_pages=F.dense(k_pages, k_scale, None), v_pages=F.dense(v_pages, v_scale, None))
        R.check_attention(c, out, lse)
