"""attn_shared_prefix_paged where a part of a row's tokens weighs nothing (lse = -inf) or holds a NaN: the join of
the two parts against the 64-bit definition and attn_chunk_paged, through every kernel's epilogue and both merges."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from tests import chunk_ref as R
from tests import fp4_ref as F
from tests.test_gpu_shared_prefix import FORMATS, run, shared_case

pytestmark = pytest.mark.gpu
DEV = "cuda"
NINF, NAN = -math.inf, math.nan
# of each KV head, what its prefix and each sequence's own tokens score: every token -inf, one token NaN, or
# finite (None)
PARTS = [(NAN, NINF), (NINF, NAN), (NINF, NINF), (None, NINF), (NINF, None), (None, None), (NAN, NAN)]
P = 128
# groups of two heads; bounds on the rows choose the kernel
CASES = {
    "few rows": ([(1, 5), (1, 70), (1, 1)], dict(max_q_len=1, max_group_rows=3)),
    "two sets of rows": ([(9, 9), (12, 80)], dict(max_q_len=12, max_group_rows=21)),
    "tensor cores": ([(20, 25), (33, 100)], {}),
    "few rows, cut": ([(1, 600)], dict(max_q_len=1, max_group_rows=1)),
    "few rows, cut in many": ([(1, 4000)], dict(max_q_len=1, max_group_rows=1)),
    "tensor cores, cut": ([(20, 600)], {}),
    "tensor cores, cut in many": ([(20, 4000)], {}),
}


def set_part(c, b, lo, hi, g, kind):
    """Scores of sequence b's tokens lo .. hi - 1 of KV head g (q's first dim is 1)."""
    table, L = c["block_table"].cpu(), c["k_pages"].shape[2]
    for t in range(lo, hi if kind == NINF else lo + 1):
        c["k_pages"][int(table[b, t // L]), g, t % L, 0] = kind


def same_as_definition(c, out, lse):
    ro, rl, _ = R.attend(c["dense"])
    bad = torch.isnan(rl)
    assert torch.equal(torch.isnan(lse).cpu(), bad), "NaN among lse"
    assert torch.equal(torch.isnan(out).any(-1).cpu(), bad) and torch.equal(torch.isnan(out).all(-1).cpu(), bad), "NaN among out"
    R.check_attention(c["dense"], out, lse)  # the other rows


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("d", [64, 128])
def test_parts_without_weight_and_nan(name, d):
    members, kw = CASES[name]
    Hkv = len(PARTS)
    c = shared_case("bf16", d, [(P, members)], 2 * Hkv, Hkv, seed=21)
    c["q"][..., 0] = 1.0
    for g, (prefix, own) in enumerate(PARTS):
        if prefix is not None:
            set_part(c, 0, 0, P, g, prefix)
        if own is not None:
            for b, (_, m) in enumerate(members):
                set_part(c, b, P, P + m, g, own)
    out, lse = run(c, **kw)
    same_as_definition(c, out, lse)
    want, want_lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                          max_q_len=kw.get("max_q_len"))
    assert torch.equal(torch.isnan(lse), torch.isnan(want_lse)) and torch.equal(lse == NINF, want_lse == NINF)
    assert torch.equal(torch.isnan(out), torch.isnan(want))


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("rows", [1, 5, 12, 40])
def test_nan_in_the_prefix_of_rows_without_own_tokens(fmt, d, rows):
    """New tokens past the capacity of the table: what they see is the prefix alone, with a NaN in one KV head."""
    c = shared_case(fmt, d, [(P, [(rows, rows), (1, 1)])], 4, 2, seed=22)
    c["block_table"] = c["dense"]["block_table"] = c["block_table"][:, :P // 64].contiguous()
    c["seq_lens"] += 7
    page = int(c["block_table"][0, 1])
    if fmt == "bf16":
        c["k_pages"][page, 1, 5, 3] = NAN
    elif fmt == "fp8":
        c["k_pages"].view(torch.uint8)[page, 1, 5, 3] = 0x7F
    else:
        c["k_scale"].view(torch.uint8)[page, 1, 5, 2] = 0x7F
        F.with_dense(c)
    same_as_definition(c, *run(c, max_q_len=rows, max_group_rows=rows + 1))


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("name", ["few rows", "two sets of rows", "tensor cores", "few rows, cut", "tensor cores, cut"])
@pytest.mark.parametrize("heavy", ["prefix", "own"])
def test_values_that_are_no_numbers_under_weights_of_zero(fmt, d, name, heavy):
    """A NaN or an infinity among the values of the part that the other one outweighs by all that fp32 can tell: the
    row holds no number there, as attn_chunk_paged's, and the dims beside it do."""
    members, kw = CASES[name]
    c = shared_case(fmt, d, [(P, members)], 4, 2, seed=23)
    # one key in four dims for each part: scores +-200 apart whatever the rest of the row adds
    c["q"].zero_()
    c["q"][..., :4] = 30.0 * math.sqrt(d) / 4
    table, L = c["block_table"].cpu(), 64
    for b, (_, m) in enumerate(members):
        for i in range(-(-(P + m) // L)):
            page, up = int(table[b, i]), (i * L < P) == (heavy == "prefix")
            if fmt == "bf16":
                c["k_pages"][page, ..., :4] = 4.0 if up else -4.0
            elif fmt == "fp8":
                c["k_pages"].view(torch.uint8)[page, ..., :4] = 0x48 if up else 0xC8  # +-4
                c["k_scale"][page] = 1.0
            else:
                c["k_pages"].view(torch.uint8)[page, ..., :2] = 0x66 if up else 0xEE  # +-4
                c["k_scale"].view(torch.uint8)[page] = 0x38  # 1
    light = int(table[0, 0 if heavy == "own" else P // L])
    if fmt == "bf16":
        c["v_pages"][light, 0, 0, 7] = NAN
        c["v_pages"][light, 1, 0, 9] = math.inf
    elif fmt == "fp8":
        c["v_pages"].view(torch.uint8)[light, :, 0, 7] = 0x7F
    else:
        c["v_scale"].view(torch.uint8)[light, :, 0, 0] = 0x7F
    out, lse = run(c, **kw)
    want, want_lse = skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                          max_q_len=kw.get("max_q_len"), **F.pages_of(c))
    first = slice(0, members[0][0])
    n = members[0][0] if heavy == "own" else 1  # the light token is the prefix's first, or the first own one
    assert not torch.isfinite(want[:n]).all(-1).any(), "attn_chunk_paged"
    assert torch.equal(torch.isfinite(out[first]), torch.isfinite(want[first]))
    # five roundings of numbers of the lse's size a side: the score's two, the sum's logarithm added, ln 2, the join
    assert torch.isfinite(lse).all() and ((lse - want_lse).abs() <= 10 * 2.0 ** -24 * want_lse.abs()).all()
