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


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_nan_that_is_seen_is_told(kind, d, kernel):
    """A NaN key makes every row that sees it NaN, through one piece or many, and no other."""
    n, m = [6, 4, 2], [70, 40, 9000]
    c = R.make_case(n, m, 8, 2, d, fp8=kind == "fp8", seed=19, device=DEV)
    for b, t in ((0, 5), (2, 8000)):
        page = int(c["block_table"][b, t // 64])
        c["k_pages"].view(torch.uint8 if kind == "fp8" else torch.int16)[page, 1, t % 64] = 0x7F if kind == "fp8" else 0x7FC0
    out, lse = run(c, kernel)
    cu = c["cu_q"].tolist()
    for b in range(3):
        rows = slice(cu[b], cu[b + 1])
        assert torch.isfinite(out[rows, :4]).all() and torch.isfinite(lse[rows, :4]).all()
        hit = b != 1
        assert torch.isnan(out[rows, 4:]).all() == hit and torch.isnan(lse[rows, 4:]).all() == hit
        assert hit or torch.isfinite(out[rows]).all()


@pytest.mark.parametrize("window,n_sink", [(0, 0), (96, 3)])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_nan_where_nobody_looks(kind, d, kernel, window, n_sink):
    n, m = [5, 16, 9], [70, 300, 601]
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
    check(c, kernel, window, n_sink)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("kernel", KERNELS)
def test_fp8_scales_of_any_size(kernel, size):
    """Tiny and huge V scales, and blocks that differ by many powers of ten."""
    c = R.make_case([4, 8], [700, 300], 8, 2, 128, fp8=True, seed=25, device=DEV)
    c["v_scale"] *= size
    for spread in (False, True):
        if spread:
            g = torch.Generator().manual_seed(2)
            c["v_scale"] *= 10.0 ** torch.randint(-6, 1, c["v_scale"].shape, generator=g).to(DEV)
        out, lse = run(c, kernel)
        ro, rl, total = R.attend(c)
        out = out.cpu().double()
        big = total > 1e-36  # (bf16 and fp32 sums end at 2^-126)
        # half a step of a weight, 2^-11 for scores off by 2.5e-4, and of fp16 weights what test_gpu_chunk_fp8 counts
        tol = (WEIGHT[kernel] + 2.0 ** -11) * total + 2.0 ** -8 * ro.abs() + 2.0 ** -20 * total.amax(-1, keepdim=True)
        assert ((out - ro).abs() <= tol)[big].all() and torch.isfinite(out).all()
        assert (lse.cpu().double() - rl).abs().max() <= 6.5e-4


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fp8", [False, True])
def test_entries_outside_the_cache(fp8, kernel):
    """Table entries outside the cache: never read behind the window, zeros where seen; scales of
    blocks that nobody sees are not read either."""
    n = [5, 7]
    far = lambda b, lo, hi: hi > [500, 800][b] - n[b] - 100 or lo == 0  # noqa: E731
    c = R.make_case(n, [500, 800], 8, 2, 128, fp8=fp8, seed=8, device=DEV, held=far)
    check(c, kernel, window=90, n_sink=4)
    c["block_table"][0, 3] = 10 ** 6
    check(c, kernel, window=90, n_sink=4)
    check(c, kernel)  # every entry is seen now: those outside read zeros
    if fp8:
        spare = torch.ones(c["k_scale"].shape[0], dtype=torch.bool)
        spare[c["block_table"].cpu().long()[c["block_table"].cpu() >= 0].clamp_max(len(spare) - 1)] = False
        for s in ("k_scale", "v_scale"):
            c[s][spare.to(DEV)] = math.nan
        check(c, kernel, window=90, n_sink=4)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_rows_of_no_sequence_are_left_alone(kind, d, kernel):
    """Rows before the first sequence and behind the last, whatever they hold."""
    c = R.make_case([3, 20], [90, 300], 8, 2, d, fp8=kind == "fp8", seed=6, device=DEV, spare_rows=9)
    c["cu_q"][0] = 1
    T = c["q"].shape[0]
    c["q"][0] = math.nan
    c["q"][23:] = math.inf
    out = torch.full((T, 8, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, 8), 7.0, device=DEV)
    run(c, kernel, out=out, lse=lse)
    R.check_attention(c, out, lse)
    for spare in (slice(0, 1), slice(23, T)):
        assert (out[spare] == 7).all() and (lse[spare] == 7).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_strides(kind, d, kernel):
    c = R.make_case([1, 40, 17], [200, 90, 400], 8, 2, d, fp8=kind == "fp8", seed=9, device=DEV)
    T = c["q"].shape[0]
    wide = torch.full((T, 12, d + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:11, :d] = c["q"]
    plain = run(c, kernel)
    step = 16 if kind == "fp8" else 8
    strided = dict(c)
    for x in ("k_pages", "v_pages"):  # token-major pages with a gap behind each head
        n, h, L, _ = c[x].shape
        big = torch.zeros(n, L, h + 1, d + step, device=DEV).to(c[x].dtype)
        view = big[:, :, :h, :d].permute(0, 2, 1, 3)
        view.copy_(c[x])
        strided[x] = view
    for a, b in zip(plain, run(strided, kernel, q=wide[:, 3:11, :d])):
        assert torch.equal(a, b)
    heads_first = c["q"].transpose(0, 1).contiguous().transpose(0, 1)
    for a, b in zip(plain, run(c, kernel, q=heads_first)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_long_histories_and_a_callers_workspace(kind, d, kernel):
    """Few rows over many tiles, cut into many pieces whose partials lie in a workspace of NaN: nothing
    of it is read unwritten; twice the same bits."""
    c = R.make_case([4, 1, 7], [20000, 63, 9001], 4, 1, d, fp8=kind == "fp8", seed=11, device=DEV)
    for window, n_sink in ((0, 0), (7000, 5)):
        ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device=DEV)
        first = check(c, kernel, window, n_sink, workspace=ws)
        for a, b in zip(first, run(c, kernel, window, n_sink)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_32_bits(fp8, kernel):
    """Pages whose element offsets pass 2^31, and whose byte offsets pass 2^32 or 2^31."""
    Hkv, L, d = 8, 64, 128
    n_pages = (1 << 31) // (Hkv * L * d) + 40
    c = R.make_case([4, 7], [100, 130], 32, Hkv, d, fp8=fp8, seed=17, device=DEV)
    n = c["k_pages"].shape[0]
    far = dict(c, block_table=torch.where(c["block_table"] < 0, -1, c["block_table"] + n_pages - n).to(torch.int32))
    for x in ("k_pages", "v_pages"):
        far[x] = torch.empty(n_pages, Hkv, L, d, dtype=c[x].dtype, device=DEV)
        far[x].view(torch.uint8)[n_pages - n:] = c[x].view(torch.uint8)
    if fp8:
        for x in ("k_scale", "v_scale"):
            far[x] = torch.zeros(n_pages, Hkv, 1, device=DEV)
            far[x][n_pages - n:] = c[x]
    for a, b in zip(check(c, kernel), run(far, kernel)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind,d", TYPES)
def test_two_graphs_and_an_eager_call(kind, d, kernel):
    """Two captured calls with other windows replayed in turn for other lengths, on two streams at
    once, beside eager calls."""
    c = R.make_case([30, 1, 1, 8], [700, 700, 700, 700], 8, 2, d, fp8=kind == "fp8", seed=16, device=DEV)
    T = c["q"].shape[0]
    outs, graphs = [], []
    run(c, kernel)
    for window in (0, 100):
        o = torch.zeros(T, 8, d, dtype=torch.bfloat16, device=DEV), torch.zeros(T, 8, device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            skv.attn_chunk_paged(c["q"], c["k_pages"], c["v_pages"], c["seq_lens"], c["cu_q"], c["block_table"],
                                 max_q_len=bound(kernel, 4, T), window=window, k_scale=c["k_scale"], v_scale=c["v_scale"],
                                 out=o[0], lse=o[1])
        outs.append(o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for cu, m in (([0, 30, 31, 32, 40], [700, 3, 650, 44]), ([0, 0, 1, 39, 40], [0, 1, 500, 200]),
                  ([0, 10, 20, 30, 31], [60, 600, 33, 699])):
        c["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
        c["seq_lens"].copy_(torch.tensor(m, dtype=torch.int32))
        for o in outs:
            o[0].fill_(5.0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = run(c, kernel, window=100)
        for (out, lse), window in zip(outs, (0, 100)):
            R.check_attention(c, out, lse, window)
            assert (out[cu[-1]:] == 5).all()
        assert torch.equal(eager[0][: cu[-1]], outs[1][0][: cu[-1]])


# ------------------------------------------------------------------ many items a CTA


def rows_of_interest(n, m, Gr, window):
    """New tokens at the borders: of the chunk, of row tiles of 128 and 256 rows, of 64 and 128
    tokens, and some between."""
    per = max(1, 128 // Gr)
    rows = {0, 1, n - 1, n - 2, n // 2, n // 3}
    for t in range(per, n, per):
        if t // per % 5 in (0, 1):
            rows |= {t - 1, t}
    for p in range((m - n) // 128 * 128, m, 128 * 3):
        rows |= {p - (m - n) - 1, p - (m - n)}
    return sorted(r for r in rows if 0 <= r < n)


def check_rows(c, out, lse, window, n_sink):
    """chunk_ref.check_attention on the rows of interest alone: each as a sequence of one token."""
    Hq, Hkv = c["q"].shape[1], c["k_pages"].shape[1]
    Gr = 1 << (Hq // Hkv - 1).bit_length()
    cu, m = c["cu_q"].tolist(), c["seq_lens"].tolist()
    picks = [(b, r) for b in range(len(m)) for r in rows_of_interest(cu[b + 1] - cu[b], m[b], Gr, window)]
    rows = torch.tensor([cu[b] + r for b, r in picks])
    one = dict(c, q=c["q"][rows.to(DEV)], block_table=c["block_table"][torch.tensor([b for b, _ in picks]).to(DEV)],
               seq_lens=torch.tensor([m[b] - (cu[b + 1] - cu[b]) + r + 1 for b, r in picks]),
               cu_q=torch.arange(len(picks) + 1))
    R.check_attention(one, out[rows.to(DEV)], lse[rows.to(DEV)], window, n_sink)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (300, 70), (1000, 4)])
@pytest.mark.parametrize("G", [8, 5])
@pytest.mark.parametrize("kind,d", TYPES)
def test_many_items_a_cta(kind, d, G, window, n_sink):
    """Long ragged prompts beside decode rows: several items of more than 128 rows for each of the
    persistent CTAs, odd numbers of tiles, items of few rows between them."""
    n, m = [1700, 1, 1303, 1, 129, 1], [2300, 3001, 1303, 64, 900, 1]
    c = R.make_case(n, m, 8 * G, 8, d, fp8=kind == "fp8", seed=G + window, device=DEV)
    Gr = 8
    pairs = 8 * sum(-(-x * Gr // 256) for x in n if x * Gr > 128)
    assert pairs >= 2 * 304  # items of more than 128 rows: four and more a CTA of 152
    out, lse = run(c, "tc", window, n_sink)
    check_rows(c, out, lse, window, n_sink)
    for a, b in zip((out, lse), run(c, "tc", window, n_sink)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind,d", TYPES)
def test_many_items_in_several_pieces(kind, d):
    """As many sequences of a pair item each as there are CTAs and more, their histories cut into
    pieces: pair items whose partials are joined, with solo items among them."""
    B = 60
    n = [65 if b % 3 else 5 for b in range(B)]
    m = [n[b] + 64 * (b % 5) * 9 + 7 * b for b in range(B)]
    c = R.make_case(n, m, 16, 4, d, fp8=kind == "fp8", seed=41, device=DEV)
    for window, n_sink in ((0, 0), (200, 3)):
        out, lse = run(c, "tc", window, n_sink)
        check_rows(c, out, lse, window, n_sink)


@pytest.mark.parametrize("kernel", ["rows16", "rows32"])
@pytest.mark.parametrize("kind,d", TYPES)
def test_many_pieces_a_cta(kind, d, kernel):
    """The kernels for few rows under long chunks (a bound that is too small): several items a CTA,
    each of several tiles a warp."""
    n, m = [300, 1, 77, 0, 130], [1500, 900, 77, 64, 2000]
    for G in (4, 3):
        c = R.make_case(n, m, 4 * G, 4, d, fp8=kind == "fp8", seed=42, device=DEV)
        for window, n_sink in ((0, 0), (700, 66)):
            out, lse = run(c, kernel, window, n_sink)
            check_rows(c, out, lse, window, n_sink)
