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
