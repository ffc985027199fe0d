"""GPU tests of qk_norm_rope_append against the plain 64-bit definition, and of a layer's step
(append, then attention over the same pages)."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged
from tests import chunk_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(n, m, Hq, Hkv, d, fp8=False, seed=0, block_len=64, per_head=False, wdtype=torch.bfloat16, rot=None, spare=0):
    c = R.make_case(n, m, Hq, Hkv, d, block_len=block_len, fp8=fp8, seed=seed, device=DEV, spare_rows=spare)
    g, T = c["gen"], c["q"].shape[0]
    c["qkv"] = R.bf16(T, (Hq + 2 * Hkv) * d, gen=g, device=DEV)
    w = (1 + 0.3 * torch.randn(Hq + Hkv, d, generator=g)).to(wdtype).to(DEV)
    c["qw"], c["kw"] = (w[:Hq].contiguous(), w[Hq:].contiguous()) if per_head else (w[0].clone(), w[Hq].clone())
    rot = d if rot is None else rot
    c["cos"], c["sin"] = paged.rotation_tables(c["block_table"].shape[1] * block_len, rot, device=DEV) if rot else (None, None)
    return c


def append(c, Hq, Hkv, **kw):
    q, k, v = paged.split_qkv(c["qkv"], Hq, Hkv)
    args = dict(cos=c["cos"], sin=c["sin"], q_weight=c["qw"], k_weight=c["kw"], k_scale=c["k_scale"], v_scale=c["v_scale"])
    args.update(kw)
    out = skv.qk_norm_rope_append(q, k, v, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"], **args)
    torch.cuda.synchronize()
    return out


def close(got, want, half_step):
    """One rounding of a value computed in fp32: half a step of the value, and 2^-18 of the
    head's largest value for the fp32 arithmetic before it."""
    got, want = got.cpu().double(), want.cpu().double()
    tol = half_step * want.abs() + (2.0 ** -18 + half_step * 2.0 ** -18) * want.abs().amax(-1, keepdim=True)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol.clamp_min(1e-30)).max()


def check(c, before, q_out, Hq, Hkv, eps=1e-6, interleaved=False, positions=None, kw=()):
    """Queries, the written page rows, and every other byte of the pages."""
    kw = dict(kw)
    q, k, v = paged.split_qkv(c["qkv"], Hq, Hkv)
    where = R.places(c)
    rows = torch.tensor([r for _, _, r in where], dtype=torch.long)
    pos = torch.tensor([p for _, p, _ in where], dtype=torch.long) if positions is None else positions.cpu().long()[rows]
    tables = kw.get("cos", c["cos"]), kw.get("sin", c["sin"])
    want_q = R.norm_rope(q.cpu()[rows], kw.get("q_weight", c["qw"]), *tables, pos, eps, interleaved)
    want_k = R.norm_rope(k.cpu()[rows], kw.get("k_weight", c["kw"]), *tables, pos, eps, interleaved)
    close(q_out.cpu()[rows], want_q, 2.0 ** -8)
    L, n_pages = c["k_pages"].shape[2], c["k_pages"].shape[0]
    table = c["block_table"].cpu()
    for pages, old, want, scale in ((c["k_pages"], before[0], want_k, c["k_scale"]),
                                    (c["v_pages"], before[1], v.cpu().double()[rows], c["v_scale"])):
        bits = torch.uint8 if scale is not None else torch.int16
        kept = torch.ones(pages.shape[0], pages.shape[2], dtype=torch.bool)
        for i, (b, p, _) in enumerate(where):
            if not 0 <= p < table.shape[1] * L:
                continue
            page = int(table[b, p // L])
            if not 0 <= page < n_pages:
                continue
            kept[page, p % L] = False
            got = pages[page, :, p % L].cpu()
            if scale is None:
                close(got, want[i], 2.0 ** -8)
            else:
                s = scale[page, :, p % L // 64].cpu().double()[:, None]
                y = (want[i] / s).clamp(-448, 448)
                # half a step of e4m3 (2^-4), below 2^-6 half the subnormal step (2^-10)
                tol = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10)) + 2.0 ** -18 * y.abs().amax()
                assert ((got.double() - y).abs() <= tol).all()
        a = pages.cpu().view(bits).transpose(1, 2)[kept]
        b = old.cpu().view(bits).transpose(1, 2)[kept]
        assert torch.equal(a, b)


def go(c, Hq, Hkv, **kw):
    before = c["k_pages"].clone(), c["v_pages"].clone()
    out = append(c, Hq, Hkv, **kw)
    check(c, before, out, Hq, Hkv, kw.get("eps", 1e-6), kw.get("interleaved", False), kw.get("positions"), kw)
    assert skv.device_error() == 0
    return out


TYPES = [("bf16", 64), ("bf16", 128), ("fp8", 128)]
N, M = [1, 70, 0, 1, 33], [65, 70, 9, 1, 200]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (5, 5), (7, 1), (40, 8)])
@pytest.mark.parametrize("kind,d", TYPES)
def test_ragged_chunks(kind, d, Hq, Hkv, interleaved):
    go(make(N, M, Hq, Hkv, d, fp8=kind == "fp8", seed=Hq), Hq, Hkv, interleaved=interleaved)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind,d", TYPES)
def test_partial_rotation(kind, d, interleaved, rot):
    go(make(N, M, 6, 2, d, fp8=kind == "fp8", seed=rot, rot=rot, block_len=128), 6, 2, interleaved=interleaved)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
def test_weights(per_head, wdtype):
    for kind, d in TYPES:
        c = make(N, M, 6, 2, d, fp8=kind == "fp8", seed=4, per_head=per_head, wdtype=wdtype)
        go(c, 6, 2, eps=1e-5)
        go(c, 6, 2, q_weight=None)
        go(c, 6, 2, k_weight=None)
        go(c, 6, 2, q_weight=None, k_weight=None, cos=None, sin=None)


def test_positions_choose_the_rotation_not_the_place():
    c = make(N, M, 8, 2, 128, seed=5)
    g = torch.Generator().manual_seed(1)
    positions = torch.randint(0, c["cos"].shape[0], (c["q"].shape[0],), generator=g, dtype=torch.int32).to(DEV)
    go(c, 8, 2, positions=positions)


def test_positions_outside_the_tables_are_told():
    c = make([3], [3], 8, 2, 128, seed=6)
    positions = torch.tensor([0, c["cos"].shape[0], -1], dtype=torch.int32, device=DEV)
    out = append(c, 8, 2, positions=positions)
    assert skv.device_error() == 8
    assert skv.device_error() == 0
    assert torch.isfinite(out[0].float()).all() and torch.isnan(out[1:].float()).all()
    page = int(c["block_table"][0, 0])
    assert torch.isnan(c["k_pages"][page, :, 1:3].float()).all()
    assert torch.equal(c["v_pages"][page, :, :3].transpose(0, 1), paged.split_qkv(c["qkv"], 8, 2)[2])


@pytest.mark.parametrize("kind,d", TYPES)
def test_tokens_without_a_place_are_not_stored(kind, d):
    """Pages outside the cache, places before 0 and past the table: the query still goes out."""
    c = make([70, 4, 5], [70, 2, 66], 8, 2, d, fp8=kind == "fp8", seed=7, rot=0)
    c["block_table"][0, 0] = -1
    c["block_table"][2, 0] = 10 ** 6
    go(c, 8, 2)
    c["seq_lens"][0] = 3 * 64  # behind the last page of the table
    go(c, 8, 2)


def test_rows_of_no_sequence_are_left_alone():
    c = make([3, 20], [90, 300], 8, 2, 128, seed=8, spare=9)
    c["cu_q"][0] = 1
    out = torch.full_like(c["q"], 7.0)
    before = c["k_pages"].clone(), c["v_pages"].clone()
    append(c, 8, 2, q_out=out)
    check(c, before, out, 8, 2)
    assert (out[:1] == 7).all() and (out[23:] == 7).all()


def test_rows_past_the_batch_are_clipped():
    """A last sequence said to reach past the packed rows has those that exist, in both calls."""
    n, m, Hq, Hkv, d = [3, 6], [90, 130], 8, 2, 128
    c = make(n, m, Hq, Hkv, d, seed=13)
    far = dict(c, k_pages=c["k_pages"].clone(), v_pages=c["v_pages"].clone(), cu_q=c["cu_q"].clone())
    far["cu_q"][-1] += 7
    want, got = append(c, Hq, Hkv), append(far, Hq, Hkv)
    assert torch.equal(got, want)
    assert torch.equal(far["k_pages"], c["k_pages"]) and torch.equal(far["v_pages"], c["v_pages"])
    for x in (0, 1):  # either kernel
        a, b = (skv.attn_chunk_paged(want, y["k_pages"], y["v_pages"], y["seq_lens"], y["cu_q"], y["block_table"],
                                     max_q_len=x) for y in (c, far))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind,d", TYPES)
@pytest.mark.parametrize("n,m,Hq,Hkv", [
    ([1500, 0, 700], [1500, 3, 900], 1, 1),    # as many tokens a CTA as there can be
    ([2, 5, 1], [2, 64, 129], 40, 20),         # more KV heads than have their scales looked up early
    ([0, 1, 0, 2] * 80, [3, 70, 0, 2] * 80, 4, 2),
])
def test_head_counts_and_batches(kind, d, n, m, Hq, Hkv):
    go(make(n, m, Hq, Hkv, d, fp8=kind == "fp8", seed=14), Hq, Hkv)


def test_in_place_and_strided_outputs():
    c = make(N, M, 8, 2, 128, seed=9)
    want = append(c, 8, 2)
    wide = torch.zeros(c["q"].shape[0], 11, 136, dtype=torch.bfloat16, device=DEV)
    append(c, 8, 2, q_out=wide[:, 2:10, :128])
    assert torch.equal(wide[:, 2:10, :128], want)
    assert (wide[:, :2] == 0).all() and (wide[:, 10:] == 0).all() and (wide[..., 128:] == 0).all()
    rest = paged.split_qkv(c["qkv"].clone(), 8, 2)[1:]
    q = paged.split_qkv(c["qkv"], 8, 2)[0]
    append(c, 8, 2, q_out=q)
    assert torch.equal(q, want)
    for a, b in zip(rest, paged.split_qkv(c["qkv"], 8, 2)[1:]):
        assert torch.equal(a, b)


def test_scales_that_are_no_scales_store_zeros():
    c = make([64], [64], 8, 2, 128, fp8=True, seed=10)
    page = int(c["block_table"][0, 0])
    for bad in (0.0, -1.0, math.inf, math.nan):
        c["k_scale"][page] = bad
        append(c, 8, 2)
        assert (c["k_pages"][page].view(torch.uint8) == 0).all()
    c["v_scale"][page] = 1e-30  # everything saturates
    append(c, 8, 2)
    assert (c["v_pages"][page].float().abs() == 448).all()


def test_strided_pages():
    for kind, d in TYPES:
        c = make(N, M, 8, 2, d, fp8=kind == "fp8", seed=11)
        step = 16 if kind == "fp8" else 8
        for x in ("k_pages", "v_pages"):
            n, h, L, _ = c[x].shape
            big = torch.zeros(n, L, h + 1, d + step, device=DEV).to(c[x].dtype)
            view = big[:, :, :h, :d].permute(0, 2, 1, 3)
            view.copy_(c[x])
            c[x] = view
        before = c["k_pages"].clone(), c["v_pages"].clone()
        out = append(c, 8, 2)
        flat = dict(c, k_pages=c["k_pages"].contiguous(), v_pages=c["v_pages"].contiguous())
        check(flat, (before[0].contiguous(), before[1].contiguous()), out, 8, 2)


def test_pages_past_32_bits():
    Hkv, L, d = 8, 64, 128
    n_pages = (1 << 31) // (Hkv * L * d) + 8
    c = make([70], [70], 16, Hkv, d, seed=12)
    k = torch.zeros(n_pages, Hkv, L, d, dtype=torch.bfloat16, device=DEV)
    far = dict(c, k_pages=k, v_pages=torch.zeros_like(k),
               block_table=torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device=DEV))
    append(c, 16, Hkv)
    append(far, 16, Hkv)
    for x in ("k_pages", "v_pages"):
        for i, n in ((0, 64), (1, 6)):
            assert torch.equal(far[x][n_pages - 1 - 2 * i, :, :n], c[x][int(c["block_table"][0, i]), :, :n])


# ------------------------------------------------------------------ a layer's step


@pytest.mark.parametrize("window,n_sink", [(0, 0), (80, 2)])
@pytest.mark.parametrize("kind,d", TYPES)
def test_chunk_step(kind, d, window, n_sink):
    """Prompts in two chunks, then decode steps: every step against the definition over the
    pages as they stand, and all of it captured once and replayed."""
    Hq, Hkv, B, cap = 8, 2, 3, 256
    g = torch.Generator().manual_seed(21)
    T = 64
    c = make([1] * B, [cap] * B, Hq, Hkv, d, fp8=kind == "fp8", seed=22)
    c["qkv"] = R.bf16(T, (Hq + 2 * Hkv) * d, gen=g, device=DEV)
    out = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(T, Hq, device=DEV)
    kw = dict(cos=c["cos"], sin=c["sin"], q_weight=c["qw"], k_weight=c["kw"], k_scale=c["k_scale"], v_scale=c["v_scale"],
              window=window, n_sink=n_sink, out=out, lse=lse)
    args = (c["qkv"], Hq, Hkv, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"])
    paged.chunk_step(*args, **kw)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        paged.chunk_step(*args, **kw)
    held = [0] * B
    for n in ([30, 0, 34], [30, 20, 1], [1, 44, 1], [1, 1, 1], [0, 1, 1]):
        held = [h + x for h, x in zip(held, n)]
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        c["qkv"].copy_(R.bf16(T, (Hq + 2 * Hkv) * d, gen=g, device=DEV))
        c["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
        c["seq_lens"].copy_(torch.tensor(held, dtype=torch.int32))
        before = c["k_pages"].clone(), c["v_pages"].clone()
        graph.replay()
        torch.cuda.synchronize()
        assert skv.device_error() == 0
        q, k, v = paged.split_qkv(c["qkv"], Hq, Hkv)
        again = append(c, Hq, Hkv)  # the same bytes again
        check(c, before, again, Hq, Hkv)
        R.check_attention(c, out, lse, window, n_sink, q=again)


def test_chunk_step_equals_the_paged_decode():
    """A decode step of equal lengths against the fused paged decode call on the same pages."""
    Hq, Hkv, d, B = 16, 2, 128, 4
    c = make([1] * B, [300] * B, Hq, Hkv, d, seed=23)
    out, lse = paged.chunk_step(c["qkv"], Hq, Hkv, c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                cos=c["cos"], sin=c["sin"], q_weight=c["qw"], k_weight=c["kw"], max_q_len=1)
    q = append(c, Hq, Hkv)
    bounds = torch.tensor([[0, 320]] * B, dtype=torch.int32, device=DEV)
    ro, rl = skv.gqa_decode_attn_paged(q.view(B, 1, Hq, d), c["k_pages"], c["v_pages"], c["seq_lens"], bounds,
                                       c["block_table"])
    torch.cuda.synchronize()
    # either is within 2^-8 (sum p|v| + |out|) of the exact value; |v| <= 5
    assert (out.float() - ro[:, 0].float()).abs().max() <= 4 * 2.0 ** -8 * 5
    assert (lse - rl[:, 0]).abs().max() <= 5e-4
