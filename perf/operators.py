"""Cases of the chunk operators over a paged KV cache: qk_norm_rope_append, which normalises and
rotates the new tokens' queries and keys and writes keys and values into the pages, and
attn_chunk_paged, attention of ragged chunks of new tokens over the pages (causal, or with a
sliding window and a few first tokens that stay visible).

``run`` does a case's operator in elementary torch operations in 32 bits, or, where ``own`` is
true, through the library's entry points.
"""

import math
import random

import torch

own = False

DEV = "cuda"
SCALE_BLOCK = 64


# ------------------------------------------------------------------ cases


def listed():
    a = dict(op="append", d=128, block_len=64, fp8=False, per_head=False, paired=False, rot=128)
    t = dict(op="attn", d=128, block_len=64, fp8=False, window=0, n_sink=0)
    return [
        # the decode step of a serving batch: one token per sequence, latency counts
        dict(a, name="append decode step", n_dec=64, n_chunk=0, chunk=0, ctx_lo=200, ctx=3000, Hq=32, Hkv=8, paired=True),
        # a prompt chunk of the ring-prefill shape entering the cache
        dict(a, name="append prompt chunk", n_dec=0, n_chunk=1, chunk=4096, ctx_lo=4096, ctx=4096, Hq=128, Hkv=8),
        # ragged chunks and decode tokens into a calibrated fp8 cache, weights of their own per
        # head, half of each head rotated
        dict(a, name="append ragged fp8", n_dec=11, n_chunk=5, chunk=2000, ctx_lo=50, ctx=3100, Hq=64, Hkv=8,
             fp8=True, per_head=True, rot=64, block_len=128),
        # the smallest call: one new token of one short sequence
        dict(t, name="one token short", n_dec=1, n_chunk=0, chunk=0, ctx_lo=1024, ctx=1024, Hq=8, Hkv=2, d=64),
        # decode of a serving batch with ragged histories
        dict(t, name="decode bf16", n_dec=64, n_chunk=0, chunk=0, ctx_lo=4096, ctx=16384, Hq=64, Hkv=8),
        # decode over long fp8 histories
        dict(t, name="decode fp8", n_dec=16, n_chunk=0, chunk=0, ctx_lo=20000, ctx=65536, Hq=128, Hkv=8, fp8=True,
             block_len=256),
        # a prompt chunk behind a long history, the ring-prefill shape
        dict(t, name="prompt chunk", n_dec=0, n_chunk=1, chunk=4096, ctx_lo=32768, ctx=32768, Hq=128, Hkv=8),
        # continuous batching: two prompt chunks among decoding sequences
        dict(t, name="mixed batch", n_dec=30, n_chunk=2, chunk=2048, ctx_lo=2048, ctx=12288, Hq=64, Hkv=8,
             block_len=128),
        # several proposed tokens per sequence checked at once, an odd group of 5 heads
        dict(t, name="draft check", n_dec=0, n_chunk=24, chunk=5, ctx_lo=300, ctx=9001, Hq=40, Hkv=8),
        # ragged prompt chunks over an fp8 cache
        dict(t, name="prompt fp8", n_dec=0, n_chunk=3, chunk=1501, ctx_lo=1501, ctx=6007, Hq=64, Hkv=8, fp8=True),
        # a long prompt chunk of a sliding-window layer with sinks
        dict(t, name="window prompt", n_dec=0, n_chunk=1, chunk=8192, ctx_lo=16384, ctx=16384, Hq=64, Hkv=8,
             window=1024, n_sink=4),
        # the same layer decoding a large batch whose pages behind the window were handed back
        dict(t, name="window decode", n_dec=128, n_chunk=0, chunk=0, ctx_lo=1000, ctx=32768, Hq=64, Hkv=8, window=4096,
             n_sink=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(Hkv=Hkv, block_len=rng.choice([64, 64, 128, 256, 320]))
    if rng.random() < 0.3:
        c.update(op="append", d=rng.choice([64, 128, 128]), Hq=Hkv * rng.choice([1, 2, 3, 5, 7, 8, 16]),
                 n_dec=rng.choice([0, 1, _log_int(rng, 2, 200)]), per_head=rng.random() < 0.3, paired=rng.random() < 0.4)
        c.update(n_chunk=0 if c["n_dec"] and rng.random() < 0.4 else rng.randint(1, 4))
        c.update(chunk=_log_int(rng, 2, 4096) if c["n_chunk"] else 0)
        c.update(fp8=c["d"] == 128 and rng.random() < 0.4, rot=c["d"] // rng.choice([1, 1, 2]))
        lo = max(1, c["chunk"])
        c.update(ctx_lo=lo, ctx=lo + _log_int(rng, 1, 2000))
        return c
    c.update(op="attn", fp8=rng.random() < 0.3)
    c.update(d=128 if c["fp8"] else rng.choice([64, 128, 128]))
    kind = rng.choice(["decode", "drafts", "chunk", "mixed"])
    G = rng.choice([1, 2, 4, 8, 8, 16, 3, 5, 6, 7])
    c.update(Hq=Hkv * G, n_dec=0, n_chunk=0, chunk=0)
    if kind == "decode":
        c.update(n_dec=_log_int(rng, 1, 128), ctx_lo=rng.randint(1, 500), ctx=_log_int(rng, 500, 16384))
    elif kind == "drafts":
        c.update(n_chunk=_log_int(rng, 1, 64), chunk=rng.randint(2, 9), ctx_lo=rng.randint(9, 500), ctx=_log_int(rng, 500, 16384))
    elif kind == "chunk":
        c.update(n_chunk=rng.randint(1, 4), chunk=_log_int(rng, 10, 2500))
        c.update(ctx_lo=c["chunk"], ctx=c["chunk"] + _log_int(rng, 1, 12000))
    else:
        c.update(n_dec=_log_int(rng, 1, 40), n_chunk=rng.randint(1, 3), chunk=_log_int(rng, 10, 2000))
        c.update(ctx_lo=c["chunk"], ctx=c["chunk"] + _log_int(rng, 1, 8000))
    w = rng.random() < 0.4
    c.update(window=_log_int(rng, 1, 4096) if w else 0, n_sink=rng.choice([0, 1, 4, 100]) if w else 0)
    return c


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: the chunks, then the decoding ones."""
    r = random.Random("%(n_dec)d %(n_chunk)d %(chunk)d %(ctx_lo)d %(ctx)d" % case)
    q = [case["chunk"] if i == 0 or case["chunk"] < 10 else r.randint(1, case["chunk"]) for i in range(case["n_chunk"])]
    q += [1] * case["n_dec"]
    s = [case["ctx"] if i == 0 else r.randint(max(case["ctx_lo"], q[i]), max(case["ctx"], q[i])) for i in range(len(q))]
    return q, s


def _reach(case, n, s):
    """(first tokens, first token of the window) that n new tokens of a history of s can see."""
    lo = max(0, s - n - case["window"] + 1) if case.get("window") else 0
    return min(case.get("n_sink", 0), lo), lo


def work(case):
    q, s = _lengths(case)
    T, Hq, Hkv, d = sum(q), case["Hq"], case["Hkv"], case["d"]
    esz = 1 if case["fp8"] else 2
    if case["op"] == "append":
        heads = case["Hq"] + case["Hkv"]
        tables = 4 * case["rot"] * T  # a row of cosines and one of sines for each token
        return {"bytes": 2 * T * d * (Hq + 2 * Hkv) + 2 * T * d * Hq + 2 * T * d * Hkv * esz + tables,
                "flops": T * d * heads * 7}
    pairs = tokens = 0
    for n, m in zip(q, s):
        w = case["window"] or m
        first, lo = _reach(case, n, m)
        tokens += first + m - lo
        for p in (range(m - n, m) if case["window"] else ()):
            pairs += min(p + 1, w) + min(case["n_sink"], max(0, p + 1 - w))
        if not case["window"]:
            pairs += n * (m - n) + n * (n + 1) // 2
    scales = 8 * tokens * Hkv // SCALE_BLOCK if case["fp8"] else 0
    return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 2 * tokens * Hkv * d * esz + scales, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ inputs


def _quantised(x):
    """e4m3 codes [.., block, d] and one scale per (page, head, 64 tokens): amax / 448."""
    n, h, b, d = x.shape
    blocks = x.float().view(n, h, b // SCALE_BLOCK, SCALE_BLOCK, d)
    scale = blocks.abs().amax((3, 4)).clamp_min(1e-6) / 448.0
    return (blocks / scale[..., None, None]).to(torch.float8_e4m3fn).view(n, h, b, d), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q_lens, seq_lens = _lengths(case)
    T, B, L = sum(q_lens), len(q_lens), case["block_len"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    # the pages that a sequence still holds: all of its own, or those of its sinks and window
    held = []
    for n, m in zip(q_lens, seq_lens):
        first, lo = _reach(case, n, m)
        held.append([i for i in range(-(-m // L)) if i * L < first or (i + 1) * L > lo])
    n_pages, width = sum(map(len, held)) + 3, max(-(-m // L) for m in seq_lens)
    shuffled = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, blocks in enumerate(held):
        for i in blocks:
            table[b, i] = shuffled.pop()
    k_pages, v_pages = randn(n_pages, Hkv, L, d), randn(n_pages, Hkv, L, d)
    k_scale = v_scale = None
    if case["fp8"]:
        (k_pages, k_scale), (v_pages, v_scale) = _quantised(k_pages), _quantised(v_pages)
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, block_table=table.to(DEV),
             seq_lens=torch.tensor(seq_lens, dtype=torch.int32, device=DEV),
             cu_q=torch.tensor([sum(q_lens[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV))
    if case["op"] == "append":
        s["qkv"] = randn(T, (Hq + 2 * Hkv) * d)  # the fused projection's output
        w = (1.0 + 0.2 * torch.randn(Hq + Hkv, d, generator=g, device=DEV)).to(torch.bfloat16)
        s["q_weight"], s["k_weight"] = (w[:Hq], w[Hq:]) if case["per_head"] else (w[0], w[Hq])
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(width * L, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    s["q"] = randn(T, Hq, d)
    s["max_q_len"] = max(q_lens)
    # sequences of one chunk length, with the longest history among them
    s["groups"] = [(n, torch.tensor([b for b in range(B) if q_lens[b] == n], device=DEV),
                    max(seq_lens[b] for b in range(B) if q_lens[b] == n)) for n in sorted(set(q_lens))]
    return s


# ------------------------------------------------------------------ the operators


def run(s):
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


def _split(s):
    """The queries, keys and values of the fused projection, as views."""
    c = s["case"]
    x = s["qkv"].view(s["qkv"].shape[0], c["Hq"] + 2 * c["Hkv"], c["d"])
    return x[:, : c["Hq"]], x[:, c["Hq"] : c["Hq"] + c["Hkv"]], x[:, c["Hq"] + c["Hkv"] :]


def _append(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        import mla_decode_attention_gqa_gb300 as skv

        q_out = skv.qk_norm_rope_append(q, k, v, s["k_pages"], s["v_pages"], s["seq_lens"], s["cu_q"], s["block_table"],
                                        cos=s["cos"], sin=s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                        eps=1e-6, interleaved=c["paired"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                        scale_block=SCALE_BLOCK)
        return {"q": q_out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    L, rot = c["block_len"], c["rot"]
    row = torch.arange(q.shape[0], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"], row, right=True) - 1
    pos = s["seq_lens"][seq] - s["cu_q"][seq + 1] + row
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]

    def norm_rope(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if c["paired"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, x[..., rot:]), -1)

    page, at = s["block_table"][seq, pos // L], pos % L
    for x, pages, scale in ((norm_rope(k, s["k_weight"]), s["k_pages"], s["k_scale"]), (v.float(), s["v_pages"], s["v_scale"])):
        if c["fp8"]:
            x = (x / scale[page, :, at // SCALE_BLOCK][..., None]).clamp(-448.0, 448.0).to(pages.dtype).view(torch.uint8)
            pages.view(torch.uint8)[page, :, at] = x
        else:
            pages[page, :, at] = x.to(pages.dtype)
    return {"q": norm_rope(q, s["q_weight"]).to(q.dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attend(s):
    c = s["case"]
    if own:
        import mla_decode_attention_gqa_gb300 as skv

        out, lse = skv.attn_chunk_paged(s["q"], s["k_pages"], s["v_pages"], s["seq_lens"], s["cu_q"], s["block_table"],
                                        max_q_len=s["max_q_len"], window=c["window"], n_sink=c["n_sink"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], scale_block=SCALE_BLOCK)
        return {"out": out, "lse": lse}
    L, Hkv, d, window, n_sink = c["block_len"], c["Hkv"], c["d"], c["window"], c["n_sink"]
    G = c["Hq"] // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)

    def gathered(pages, scale, page, at):  # [sequences, Hkv, tokens, d] in 32 bits
        x = pages.view(torch.uint8)[page, :, at].view(pages.dtype).float() if c["fp8"] else pages[page, :, at].float()
        if c["fp8"]:
            x *= scale[page, :, at // SCALE_BLOCK][..., None]
        return x.transpose(1, 2)

    for n, rows, longest in s["groups"]:
        new = torch.arange(n, device=DEV)
        token = s["cu_q"][rows].long()[:, None] + new
        pos = s["seq_lens"][rows].long()[:, None] - n + new
        if window and n_sink + window + n - 1 < longest:  # the sinks, then the chunk's window
            span = pos[:, :1] - window + 1 + torch.arange(window + n - 1, device=DEV)
            first = torch.arange(n_sink, device=DEV).expand(len(rows), n_sink)
            index = torch.cat((first, torch.where(span < n_sink, longest, span)), 1)
        else:
            index = torch.arange(longest, device=DEV).expand(len(rows), longest)
        seen = index[:, None] <= pos[..., None]
        if window:
            seen &= (index[:, None] > pos[..., None] - window) | (index[:, None] < n_sink)
        inside = index.clamp_max(longest - 1)
        page, at = s["block_table"][rows].long().gather(1, inside // L).clamp_min(0), inside % L
        q = s["q"][token].float().view(len(rows), n, Hkv, G, d).transpose(1, 2).reshape(len(rows), Hkv, n * G, d)
        p = torch.matmul(q * (1.0 / math.sqrt(d)), gathered(s["k_pages"], s["k_scale"], page, at).transpose(2, 3))
        p = p.view(len(rows), Hkv, n, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
        top = p.amax(-1, keepdim=True)
        p = p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(len(rows), Hkv, n * G, -1), gathered(s["v_pages"], s["v_scale"], page, at))
        o = o.view(len(rows), Hkv, n, G, d) / total
        out[token] = o.transpose(1, 2).reshape(len(rows), n, c["Hq"], d).to(out.dtype)
        lse[token] = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(len(rows), n, c["Hq"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _spans(s):
    """(first row, one behind the last, tokens with them) of each sequence."""
    cu, m = s["cu_q"].tolist(), s["seq_lens"].tolist()
    return [(cu[b], cu[b + 1], m[b]) for b in range(len(m))]


def _exact_append(s):
    c = s["case"]
    L, rot, half = c["block_len"], c["rot"], c["rot"] // 2
    q, k, v = (x.double() for x in _split(s))
    pos = torch.cat([torch.arange(m - (hi - lo), m) for lo, hi, m in _spans(s)]).to(DEV)
    cos, sin = s["cos"].double()[pos], s["sin"].double()[pos]
    first = torch.arange(half, device=DEV) * (2 if c["paired"] else 1)
    second = first + (1 if c["paired"] else half)

    def turned(x, weight):
        x = x / ((x**2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * weight.double()
        y = x.clone()
        y[..., first] = x[..., first] * cos[:, None] - x[..., second] * sin[:, None]
        y[..., second] = x[..., first] * sin[:, None] + x[..., second] * cos[:, None]
        return y

    pages = []
    for x, to, scale in ((turned(k, s["k_weight"]), s["k_pages"], s["k_scale"]), (v, s["v_pages"], s["v_scale"])):
        to = to.double()
        for b, (lo, hi, m) in enumerate(_spans(s)):
            for p0 in range((m - hi + lo) // L * L, m, L):  # the pages that the new tokens reach
                a, e = max(p0, m - hi + lo), min(p0 + L, m)
                page, y = int(s["block_table"][b, p0 // L]), x[hi - m + a : hi - m + e].transpose(0, 1)
                if c["fp8"]:
                    by = scale[page].double()[:, (torch.arange(a, e, device=DEV) - p0) // SCALE_BLOCK]
                    y = (y / by[..., None]).clamp(-448, 448)
                to[page, :, a - p0 : e - p0] = y
        pages.append(to)
    return {"q": turned(q, s["q_weight"]), "k_pages": pages[0], "v_pages": pages[1]}


def _exact_attend(s):
    c = s["case"]
    G, L = c["Hq"] // c["Hkv"], c["block_len"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, (lo, hi, m) in enumerate(_spans(s)):
        for r in range(lo, hi, 512):
            e = min(r + 512, hi)
            pos = torch.arange(m - hi + r, m - hi + e, device=DEV)
            start = max(0, m - hi + r - c["window"] + 1) if c["window"] else 0
            t = torch.arange(start, m - hi + e, device=DEV)
            if start:
                t = torch.cat((torch.arange(min(c["n_sink"], start), device=DEV), t))
            hidden = t[None] > pos[:, None]
            if c["window"]:
                hidden |= (pos[:, None] - t[None] >= c["window"]) & (t[None] >= c["n_sink"])
            page, at = s["block_table"][b].long()[t // L], t % L
            for h in range(c["Hkv"]):
                k, v = (x.view(torch.uint8)[page, h, at].view(x.dtype).double() if c["fp8"] else x[page, h, at].double()
                        for x in (s["k_pages"], s["v_pages"]))
                if c["fp8"]:
                    k = k * s["k_scale"][page, h, at // SCALE_BLOCK].double()[:, None]
                    v = v * s["v_scale"][page, h, at // SCALE_BLOCK].double()[:, None]
                x = torch.einsum("igd,td->igt", s["q"][r:e, h * G : (h + 1) * G].double(), k) / math.sqrt(c["d"])
                x = x.masked_fill(hidden[:, None], -math.inf)
                total = torch.logsumexp(x, -1)
                lse[r:e, h * G : (h + 1) * G] = total
                out[r:e, h * G : (h + 1) * G] = torch.einsum("igt,td->igd", torch.exp(x - total[..., None]), v)
    return {"out": out, "lse": lse}
