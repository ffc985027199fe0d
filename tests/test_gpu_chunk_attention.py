"""GPU tests of attn_chunk_paged against the plain 64-bit definition: types, head groups, ragged
chunks from one token to long ones, windows and sinks, pages that end inside a tile, rows that
see nothing, NaN where nobody looks, strides, graphs, streams and far pages."""

import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from tests import chunk_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def run(c, window=0, n_sink=0, **kw):
    out, lse = skv.attn_chunk_paged(kw.pop("q", c["q"]), c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"],
                                    c["block_table"], window=window, n_sink=n_sink, k_scale=c["k_scale"],
                                    v_scale=c["v_scale"], **kw)
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    return out, lse


def check(c, window=0, n_sink=0, **kw):
    out, lse = run(c, window, n_sink, **kw)
    R.check_attention(c, out, lse, window, n_sink, kw.get("softmax_scale"))
    return out, lse


TYPES = [("bf16", 64), ("bf16", 128), ("fp8", 128)]
MIXES = {
    "one": ([1], [1]),
    "decode": ([1, 1, 1, 1, 1], [1, 64, 65, 700, 1031]),
    "drafts": ([3, 5, 2], [129, 5, 400]),
    "chunk": ([70], [70]),
    "behind": ([129, 33], [700, 161]),
    "mixed": ([1, 150, 0, 1, 40], [333, 150, 77, 1, 640]),
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 2), (16, 1), (3, 3), (40, 8)])
@pytest.mark.parametrize("kind,d", TYPES)
def test_ragged_chunks(kind, d, Hq, Hkv, mix):
    n, m = MIXES[mix]
    c = R.make_case(n, m, Hq, Hkv, d, fp8=kind == "fp8", seed=len(mix) + Hq, device=DEV)
    check(c, max_q_len=max(n))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (5, 0), (64, 4), (100, 4), (128, 130), (300, 64), (5000, 3)])
@pytest.mark.parametrize("mix", ["decode", "drafts", "behind", "mixed"])
@pytest.mark.parametrize("kind,d", TYPES)
def test_windows_and_sinks(kind, d, mix, window, n_sink):
    n, m = MIXES[mix]
    c = R.make_case(n, m, 16, 2, d, fp8=kind == "fp8", seed=window, device=DEV)
    check(c, window, n_sink, max_q_len=max(n))


@pytest.mark.parametrize("block_len", [64, 128, 192, 320])
@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("kind,d", TYPES)
def test_page_lengths(kind, d, G, block_len):
    n, m = [1, 200, 9], [511, 450, 1000]
    c = R.make_case(n, m, 2 * G, 2, d, block_len=block_len, fp8=kind == "fp8", seed=block_len, device=DEV)
    check(c)
    check(c, window=130, n_sink=2)


@pytest.mark.parametrize("kind,d", TYPES)
def test_rows_that_see_nothing(kind, d):
    """More new tokens than cached ones (the first rows lie before position 0), no cached token
    at all, and lengths past the table's capacity."""
    c = R.make_case([7, 4, 1, 3], [3, 0, 0, 64], 8, 2, d, fp8=kind == "fp8", seed=3, device=DEV)
    check(c)
    check(c, window=2, n_sink=1)
    c["seq_lens"][1] = -5
    check(c)
    c["seq_lens"][3] = 64 + 7  # one page: tokens past it do not exist
    check(c)
    check(c, window=9, n_sink=1)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (96, 3)])
@pytest.mark.parametrize("max_q_len", [1, 16, None])
@pytest.mark.parametrize("kind,d", TYPES)
def test_nan_where_nobody_looks(kind, d, max_q_len, window, n_sink):
    n, m = ([1, 1, 1], [70, 300, 601]) if max_q_len == 1 else ([5, 16, 9], [70, 300, 601])
    c = R.make_case(n, m, 8, 2, d, fp8=kind == "fp8", seed=5, device=DEV)
    table = c["block_table"].tolist()
    used = torch.zeros(c["k_pages"].shape[0], 64, dtype=torch.bool)
    for b, (nb, mb) in enumerate(zip(n, m)):
        for t in range(mb):
            if not window or t > mb - nb - window or t < n_sink:
                used[table[b][t // 64], t % 64] = True
    hole = (~used).to(DEV)
    for x in ("k_pages", "v_pages"):
        bits = c[x].view(torch.uint8 if kind == "fp8" else torch.int16)
        bits.transpose(1, 2)[hole] = 0x7F if kind == "fp8" else 0x7FC0  # NaN
        assert torch.isnan(c[x].float()).any() or not hole.any()
    check(c, window, n_sink, max_q_len=max_q_len)


def test_scales_of_unused_pages_and_entries_outside_the_cache():
    """Table entries outside the cache: never read behind the window, zeros where seen."""
    far = lambda b, lo, hi: hi > [500, 800][b] - 100 or lo == 0  # noqa: E731
    for fp8 in (False, True):
        c = R.make_case([1, 1], [500, 800], 8, 2, 128, fp8=fp8, seed=8, device=DEV, held=far)
        check(c, window=90, n_sink=4, max_q_len=1)
        c["block_table"][0, 3] = 10 ** 6
        check(c, window=90, n_sink=4)
        check(c)  # every entry is seen now: those outside read zeros


def test_rows_of_no_sequence_are_left_alone():
    for d, fp8 in ((64, False), (128, False), (128, True)):
        c = R.make_case([3, 20], [90, 300], 8, 2, d, fp8=fp8, seed=6, device=DEV, spare_rows=9)
        c["cu_q"][0] = 1  # rows before the first sequence
        T = c["q"].shape[0]
        out = torch.full((T, 8, d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((T, 8), 7.0, device=DEV)
        run(c, out=out, lse=lse)
        R.check_attention(c, out, lse)
        for spare in (slice(0, 1), slice(23, T)):
            assert (out[spare] == 7).all() and (lse[spare] == 7).all()


@pytest.mark.parametrize("kind,d", TYPES)
def test_strided_queries_and_pages(kind, d):
    c = R.make_case([1, 40, 17], [200, 90, 400], 8, 2, d, fp8=kind == "fp8", seed=9, device=DEV)
    T = c["q"].shape[0]
    wide = torch.full((T, 12, d + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:11, :d] = c["q"]
    plain = run(c)
    step = 16 if kind == "fp8" else 8
    strided = dict(c)
    for x in ("k_pages", "v_pages"):  # token-major pages with a gap behind each head
        n, h, L, _ = c[x].shape
        big = torch.zeros(n, L, h + 1, d + step, device=DEV).to(c[x].dtype)
        view = big[:, :, :h, :d].permute(0, 2, 1, 3)
        view.copy_(c[x])
        strided[x] = view
    got = run(strided, q=wide[:, 3:11, :d])
    for a, b in zip(plain, got):
        assert torch.equal(a, b)


def test_a_contiguous_cache_is_one_page_per_sequence():
    B, Hkv, S, d = 3, 2, 320, 128
    c = R.make_case([1, 30, 4], [320, 200, 64], 8, Hkv, d, block_len=S, seed=10, device=DEV)
    g = torch.Generator().manual_seed(1)
    c["k_pages"], c["v_pages"] = (R.bf16(B, Hkv, S, d, gen=g, device=DEV) for _ in range(2))
    c["block_table"] = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    check(c)
    dec = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    q = c["q"][:3].contiguous()
    out, lse = skv.attn_chunk_paged(q, c["k_pages"], c["v_pages"], c["seq_lens"], dec, c["block_table"], max_q_len=1)
    bounds = torch.tensor([[0, S]] * B, dtype=torch.int32, device=DEV)
    ro, rl = skv.gqa_decode_attn(q.view(B, 1, 8, d), c["k_pages"], c["v_pages"], c["seq_lens"], bounds)
    assert (out.float() - ro[:, 0].float()).abs().max() <= 2.0 ** -7 * 4  # two roundings of |values| <= 4
    assert (lse - rl[:, 0]).abs().max() <= 5e-4


@pytest.mark.parametrize("kind,d", TYPES)
def test_long_histories_in_many_chunks(kind, d):
    """Single rows over many tiles: the partials of one row are dealt to several warps."""
    c = R.make_case([1, 1, 2], [20000, 63, 9001], 4, 1, d, fp8=kind == "fp8", seed=11, device=DEV)
    check(c, max_q_len=2)
    check(c, max_q_len=2, window=7000, n_sink=5)


@pytest.mark.parametrize("kind,d", TYPES)
@pytest.mark.parametrize("B", [1, 200, 700])
def test_many_sequences(kind, d, B):
    """More sequences than a block has threads."""
    n = [1 if b % 3 else 0 for b in range(B)]
    n[0] = 2
    m = [n[b] + (37 * b) % 150 for b in range(B)]
    c = R.make_case(n, m, 4, 2, d, fp8=kind == "fp8", seed=12, device=DEV)
    check(c, max_q_len=2)
    check(c, window=70, n_sink=2)


@pytest.mark.parametrize("kind,d", TYPES)
def test_large_and_falling_scores(kind, d):
    """Scores up to hundreds, rising and falling along the sequence: the running maximum moves."""
    c = R.make_case([33, 1], [500, 900], 8, 2, d, seed=13, device=DEV)
    ramp = torch.linspace(0.05, 12.0, c["k_pages"].shape[0], device=DEV)[:, None, None, None]
    c["k_pages"] = (c["k_pages"].float() * ramp).to(torch.bfloat16)
    if kind == "fp8":
        for x, s in (("k_pages", "k_scale"), ("v_pages", "v_scale")):
            c[x], c[s] = R.quantise(c[x])
    out, lse = run(c, max_q_len=33)
    ro, rl, size = R.attend(c)
    # scores of size s carry 2^-23 |s| each from the fp32 sums: e^error - 1 on every weight
    q, k = c["q"].cpu().double(), R.dense(c["k_pages"], c["k_scale"])
    most = (q.norm(dim=-1).max() * k.norm(dim=-1).max() / math.sqrt(d)).item()
    slack = 128 * 2.0 ** -23 * most
    tol = (2.0 ** -8 + slack) * (size + ro.abs()) + 2.0 ** -12 * size + 2 * slack * size
    assert ((out.cpu().double() - ro).abs() <= tol).all()
    assert (lse.cpu().double() - rl).abs().max() <= slack + 2.5e-4


def test_the_kernel_choice_does_not_change_the_result():
    for kind, d in TYPES:
        for G in (1, 5, 16):
            c = R.make_case([1, 1, 1], [900, 64, 333], 2 * G, 2, d, fp8=kind == "fp8", seed=14, device=DEV)
            for longest in (1, 3, None):
                check(c, max_q_len=longest)
            # a bound that is too small is only a worse choice
            c = R.make_case([1, 60, 1, 90], [900, 64, 333, 700], 2 * G, 2, d, fp8=kind == "fp8", seed=15, device=DEV)
            check(c, max_q_len=1)
            for window, n_sink in ((1, 0), (63, 2), (70, 65), (129, 0), (500, 130)):
                check(c, window, n_sink, max_q_len=1)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (70, 5), (700, 66)])
@pytest.mark.parametrize("Hq,Hkv,longest", [(40, 8, 5), (8, 2, 8), (17, 1, 1), (32, 1, 1), (3, 1, 10), (9, 3, 6)])
@pytest.mark.parametrize("kind,d", TYPES)
def test_two_sets_of_rows(kind, d, Hq, Hkv, longest, window, n_sink):
    """17 to 32 rows of a KV head, beside sequences of fewer (one set idle), of none and of more."""
    for seed, n, m in ((17, [longest, 1, 0, longest, 2], [1500, 1, 9, longest, 130]),
                       (18, [1, 43, longest, 20], [900, 64, 5000, 333])):
        check(R.make_case(n, m, Hq, Hkv, d, fp8=kind == "fp8", seed=seed, device=DEV), window, n_sink, max_q_len=longest)


@pytest.mark.parametrize("kind,d", TYPES)
def test_a_captured_graph_follows_the_lengths(kind, d):
    """One graph replayed for other lengths, chunk borders and tables, eager calls in between."""
    c = R.make_case([30, 1, 1, 8], [700, 700, 700, 700], 8, 2, d, fp8=kind == "fp8", seed=16, device=DEV)
    out = torch.zeros(c["q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(c["q"].shape[:2], device=DEV)
    args = (c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"])
    kw = dict(k_scale=c["k_scale"], v_scale=c["v_scale"], out=out, lse=lse)
    skv.attn_chunk_paged(*args, **kw)
    graphs = []
    for window in (0, 100):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            skv.attn_chunk_paged(*args, window=window, **kw)
        graphs.append((window, g))
    for cu, m in (([0, 30, 31, 32, 40], [700, 3, 650, 44]), ([0, 0, 1, 39, 40], [0, 1, 500, 200]),
                  ([0, 10, 20, 30, 31], [60, 600, 33, 699])):
        c["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
        c["seq_lens"].copy_(torch.tensor(m, dtype=torch.int32))
        for window, g in graphs:
            out.fill_(5.0)
            lse.fill_(5.0)
            g.replay()
            torch.cuda.synchronize()
            R.check_attention(c, out, lse, window)
            assert (out[cu[-1]:] == 5).all()


def test_two_streams_at_once():
    cases = [R.make_case([1] * 8, [3000 + 100 * b for b in range(8)], 16, 2, 128, seed=20 + i, device=DEV) for i in range(2)]
    want = [run(c, max_q_len=1) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"],
                                                   c["block_table"], max_q_len=1))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_the_same_call_gives_the_same_bits():
    for d, fp8, longest in ((128, False, 1), (128, False, None), (128, True, 1), (64, False, None)):
        c = R.make_case([1] * 6, [5000, 1, 777, 64, 3000, 129], 16, 2, d, fp8=fp8, seed=30, device=DEV)
        a = run(c, max_q_len=longest)
        for _ in range(3):
            b = run(c, max_q_len=longest)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("longest", [1, None])
def test_pages_past_32_bits(longest):
    """Pages whose element offsets pass 2^31."""
    Hkv, L, d = 8, 64, 128
    n_pages = (1 << 31) // (Hkv * L * d) + 40
    c = R.make_case([1, 1], [100, 130], 16, Hkv, d, seed=17, device=DEV)
    small = c["k_pages"], c["v_pages"]
    pool = torch.empty(n_pages, Hkv, L, d, dtype=torch.bfloat16, device=DEV)
    shift = n_pages - small[0].shape[0]
    far = dict(c, block_table=torch.where(c["block_table"] < 0, -1, c["block_table"] + shift).to(torch.int32))
    want = run(c, max_q_len=longest)
    pool[shift:] = small[0]
    far["k_pages"] = pool
    far["v_pages"] = torch.empty_like(pool)
    far["v_pages"][shift:] = small[1]
    got = run(far, max_q_len=longest)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_no_rows_and_a_caller_workspace():
    c = R.make_case([4, 1], [70, 200], 8, 2, 128, seed=18, device=DEV)
    out, lse = skv.attn_chunk_paged(c["q"][:0], c["k_pages"], c["v_pages"], c["seq_lens"], torch.zeros_like(c["cu_q"]),
                                    c["block_table"])
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    want = run(c)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)  # NaN bits: nothing of it is read unwritten
    got = run(c, workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(skv.SplitKVError) as e:
        run(c, workspace=ws[:256])
    assert e.value.status == skv.SKV_EWORKSPACE


@pytest.mark.parametrize("longest", [1, None])
@pytest.mark.parametrize("kind,d", TYPES)
def test_nan_that_is_seen_is_told(kind, d, longest):
    """A NaN key makes every row that sees it NaN, through one chunk or many."""
    n, m = ([1, 1, 1], [70, 40, 9000]) if longest == 1 else ([3, 2, 1], [70, 40, 9000])
    c = R.make_case(n, m, 8, 2, d, fp8=kind == "fp8", seed=19, device=DEV)
    for b, t in ((0, 5), (2, 8000)):
        page = int(c["block_table"][b, t // 64])
        c["k_pages"].view(torch.uint8 if kind == "fp8" else torch.int16)[page, 1, t % 64] = 0x7F if kind == "fp8" else 0x7FC0
    out, lse = run(c, max_q_len=longest)
    cu = c["cu_q"].tolist()
    for b in range(3):
        rows = slice(cu[b], cu[b + 1])
        assert torch.isfinite(out[rows, :4]).all() and torch.isfinite(lse[rows, :4]).all()
        hit = b != 1
        assert torch.isnan(out[rows, 4:]).all() == hit and torch.isnan(lse[rows, 4:]).all() == hit
        assert hit or torch.isfinite(out[rows]).all()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (100, 1), (128, 1), (136, 1)])
@pytest.mark.parametrize("kind,d", TYPES)
def test_head_groups(kind, d, Hq, Hkv):
    """Groups padded to a power of two (fewer heads than a box among them), a group that fills a
    query tile alone, and one larger than that."""
    c = R.make_case([1, 9, 30], [200, 9, 150], Hq, Hkv, d, fp8=kind == "fp8", seed=Hq, device=DEV)
    check(c)
    check(c, window=40, n_sink=3)


@pytest.mark.parametrize("longest", [1, None])
def test_every_e4m3_code(longest):
    """Each code as a key element against a one-hot query: the lse of a row that sees only that
    token is the score itself; and as a value: its product is the output."""
    d, L = 128, 64
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    n = len(codes)
    k = torch.zeros(n, 1, L, d, dtype=torch.uint8)
    k[:, 0, 0, 77] = codes
    v = torch.zeros(n, 1, L, d, dtype=torch.uint8)
    v[:, 0, 0] = codes[:, None]
    value = codes.view(R.E4M3).double()
    # sequences of two tokens that see only their own (window 1): rows at position 0 and 1
    q = torch.zeros(2 * n, 1, d, dtype=torch.bfloat16)
    q[:, :, 77] = 1.0
    scale = torch.full((n, 1, 1), 0.25)
    c = dict(q=q.to(DEV), k_pages=k.view(R.E4M3).to(DEV), v_pages=v.view(R.E4M3).to(DEV), k_scale=scale.to(DEV),
             v_scale=scale.to(DEV), block_table=torch.arange(n, dtype=torch.int32, device=DEV).view(n, 1),
             seq_lens=torch.full((n,), 2, dtype=torch.int32, device=DEV),
             cu_q=torch.arange(n + 1, dtype=torch.int32, device=DEV) * 2)
    out, lse = run(c, window=1, max_q_len=longest, softmax_scale=1.0)
    got_lse, got = lse[0::2, 0].cpu().double(), out[0::2, 0].cpu().double()
    want = value * 0.25
    assert (got_lse - want).abs().max() <= 112 * 2.0 ** -22  # the base-2 scaling there and back
    assert ((got - want[:, None]).abs() <= 2.0 ** -8 * want.abs()[:, None]).all()
    assert (lse[1::2].abs() <= 1e-6).all() and (out[1::2] == 0).all()


def test_scales_of_blocks_that_nobody_sees():
    """NaN scales of blocks without a visible token, in pages that are read for others."""
    c = R.make_case([1, 40, 1], [70, 450, 700], 8, 2, 128, block_len=192, fp8=True, seed=24, device=DEV)
    for window, n_sink in ((0, 0), (100, 3)):
        x = dict(c, k_scale=c["k_scale"].clone(), v_scale=c["v_scale"].clone())
        seen = torch.zeros(c["k_scale"].shape[0], 3, dtype=torch.bool)
        table = c["block_table"].tolist()
        for b, (n, m) in enumerate(((1, 70), (40, 450), (1, 700))):
            for t in range(m):
                if not window or t > m - n - window or t < n_sink:
                    seen[table[b][t // 192], t % 192 // 64] = True
        for s in ("k_scale", "v_scale"):
            x[s].transpose(1, 2)[~seen.to(DEV)] = math.nan
        for longest in (1, None):
            out, lse = run(x, window, n_sink, max_q_len=longest)
            R.check_attention(c, out, lse, window, n_sink)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("longest", [1, None])
def test_fp8_scales_of_any_size(longest, size):
    """Tiny and huge V scales, and blocks that differ by many powers of ten: the weights keep
    their bits."""
    c = R.make_case([1, 5], [700, 300], 8, 2, 128, fp8=True, seed=25, device=DEV)
    c["v_scale"] *= size
    for spread in (False, True):
        if spread:
            g = torch.Generator().manual_seed(2)
            c["v_scale"] *= 10.0 ** torch.randint(-6, 1, c["v_scale"].shape, generator=g).to(DEV)
        out, lse = run(c, max_q_len=longest)
        ro, rl, total = R.attend(c)
        out = out.cpu().double()
        big = total > 1e-36  # (bf16 and fp32 sums end at 2^-126)
        tol = 2.0 ** -8 * (total + ro.abs()) + 2.0 ** -12 * total
        assert ((out - ro).abs() <= tol)[big].all() and torch.isfinite(out).all()
        assert (lse.cpu().double() - rl).abs().max() <= 2.5e-4
