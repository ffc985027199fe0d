"""Plain 64-bit definitions of the chunk operators, on the CPU, and seeded inputs for them."""

import math

import torch

E4M3 = torch.float8_e4m3fn


def bf16(*shape, gen, device):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16).to(device)


def quantise(x):
    """e4m3 codes and one scale per (page, head, 64 tokens): amax / 448."""
    n, h, b, d = x.shape
    blk = x.float().view(n, h, b // 64, 64, d)
    scale = blk.abs().amax((3, 4)).clamp_min(1e-6) / 448.0
    return (blk / scale[..., None, None]).to(E4M3).view(n, h, b, d), scale.contiguous()


def make_case(q_lens, seq_lens, Hq, Hkv, d, block_len=64, fp8=False, seed=0, device="cpu", spare_rows=0, held=None):
    """Packed queries, shuffled pages and tables; held(b, first token, one behind the last) says
    which pages exist (the others' table entries are -1)."""
    g = torch.Generator().manual_seed(seed)
    B = len(q_lens)
    width = max(1, max(-(-s // block_len) for s in seq_lens))
    own = [[i for i in range(-(-s // block_len)) if held is None or held(b, i * block_len, (i + 1) * block_len)]
           for b, s in enumerate(seq_lens)]
    n_pages = sum(map(len, own)) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        for i in own[b]:
            table[b, i] = order.pop()
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    c = dict(q=bf16(cu[-1] + spare_rows, Hq, d, gen=g, device=device),
             k_pages=bf16(n_pages, Hkv, block_len, d, gen=g, device=device),
             v_pages=bf16(n_pages, Hkv, block_len, d, gen=g, device=device), k_scale=None, v_scale=None,
             block_table=table.to(device), seq_lens=torch.tensor(seq_lens, dtype=torch.int32, device=device),
             cu_q=torch.tensor(cu, dtype=torch.int32, device=device), gen=g)
    if fp8:
        c["k_pages"], c["k_scale"] = quantise(c["k_pages"])
        c["v_pages"], c["v_scale"] = quantise(c["v_pages"])
    return c


def dense(pages, scale):
    x = pages.cpu().double()
    if scale is not None:
        x = x * scale.cpu().double().repeat_interleave(64, 2)[..., None]
    return x


def attend(c, window=0, n_sink=0, scale=None, q=None):
    """(out, lse, sum of p |v|) in 64 bits; rows of no sequence are NaN."""
    q = (c["q"] if q is None else q).cpu().double()
    k_pages, v_pages = dense(c["k_pages"], c["k_scale"]), dense(c["v_pages"], c["v_scale"])
    T, Hq, d = q.shape
    Hkv, L = k_pages.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, size = torch.full((T, Hq, d), math.nan, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    cu, table = c["cu_q"].tolist(), c["block_table"].cpu().long()
    for b, m in enumerate(c["seq_lens"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        if hi <= lo:
            continue
        pos = torch.arange(m - (hi - lo), m)
        t = torch.arange(max(0, min(m, table.shape[1] * L)))
        seen = t[None] <= pos[:, None]
        if window:
            seen &= (t[None] > pos[:, None] - window) | (t[None] < n_sink)
        t, seen = t[seen.any(0)], seen[:, seen.any(0)]  # what nobody sees is not read
        page, at = table[b][t // L], t % L
        real = ((page >= 0) & (page < k_pages.shape[0]))[:, None]
        for g in range(Hkv):
            k = torch.where(real, k_pages[page.clamp(0, k_pages.shape[0] - 1), g, at], 0.0)
            v = torch.where(real, v_pages[page.clamp(0, k_pages.shape[0] - 1), g, at], 0.0)
            x = torch.einsum("nhd,td->nht", q[lo:hi, g * G:(g + 1) * G], k) * scale
            x = x.masked_fill(~seen[:, None], -math.inf)
            z = torch.logsumexp(x, -1) if t.numel() else torch.full(x.shape[:2], -math.inf, dtype=torch.float64)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            out[lo:hi, g * G:(g + 1) * G] = torch.einsum("nht,td->nhd", p, v)
            size[lo:hi, g * G:(g + 1) * G] = torch.einsum("nht,td->nhd", p, v.abs())
            lse[lo:hi, g * G:(g + 1) * G] = z
    return out, lse, size


def check_attention(c, out, lse, window=0, n_sink=0, scale=None, q=None):
    """Weights are rounded to bf16 (or, times the fp8 block scale, to fp16) once and so is the
    output: |error| <= 2^-8 sum p|v| + 2^-8 |out|, with 2^-12 of sum p|v| for the fp32 sums and
    the 2^-22 exponentials.  The lse is a sum of exact products in fp32: d = 128 additions of
    terms whose absolute sum is below 16 (normal queries and keys times 1/sqrt(d)), each off by
    2^-23 of that at most: 2.5e-4."""
    ro, rl, size = attend(c, window, n_sink, scale, q)
    some = ~torch.isnan(rl)
    out, lse = out.cpu().double(), lse.cpu().double()
    tol = 2.0 ** -8 * (size + ro.abs()) + 2.0 ** -12 * size + 1e-30
    worst = ((out - ro).abs() / tol)[some]
    assert torch.isfinite(out[some]).all()
    assert worst.numel() == 0 or worst.max() <= 1.0, f"out off by {worst.max():.3g} of the tolerance"
    empty = some & (rl == -math.inf)
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    full = some & ~empty
    assert full.sum() == 0 or (lse - rl)[full].abs().max() <= 2.5e-4, (lse - rl)[full].abs().max()


def norm_rope(x, weight, cos, sin, pos, eps, interleaved):
    """x [T,H,d] in 64 bits; cos / sin tables or None."""
    x = x.cpu().double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.cpu().double()
    if cos is None:
        return x
    half = cos.shape[1]
    c, s = cos.cpu().double()[pos][:, None], sin.cpu().double()[pos][:, None]
    y = x.clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def places(c):
    """(sequence, place in it) of each packed row that belongs to a sequence."""
    cu = c["cu_q"].tolist()
    return [(b, m - (cu[b + 1] - cu[b]) + i, cu[b] + i) for b, m in enumerate(c["seq_lens"].tolist())
            for i in range(cu[b + 1] - cu[b])]
