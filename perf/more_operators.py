"""Cases of the operators that keep a paged KV cache small and read it once: qk_norm_rope_append and
attn_chunk_paged over 4-bit pages that are quantised as they are written, kv_read_paged, which reads a
cache back, and attn_shared_prefix_paged, attention of sequences whose first pages are the same.

4-bit pages hold e2m1 codes, two a byte (the even dim in the low half), an e4m3 scale for each 16 dims
of a token's head and an fp32 scale for each KV head: value = code * scale * head scale.

``run`` does a case's operator in elementary torch operations in 32 bits, or, where ``own`` is
true, through the library's entry points.
"""

import math
import random

import torch

own = False

DEV = "cuda"
SCALE_BLOCK = 64  # tokens of an fp8 scale
BLOCK = 16        # dims of a 4-bit scale


# ------------------------------------------------------------------ cases


def listed():
    a = dict(op="append", fmt="fp4", d=128, block_len=64, per_head=False, paired=False, rot=128)
    r = dict(op="read", d=128, block_len=64)
    t = dict(op="attn", fmt="fp4", d=128, block_len=64, window=0, n_sink=0)
    s = dict(op="shared", fmt="bf16", d=128, block_len=64)
    return [
        # the decode step of a serving batch, one token a sequence: latency counts
        dict(a, name="append decode step", n_dec=64, n_chunk=0, chunk=0, ctx_lo=50, ctx=400, Hq=64, Hkv=8, paired=True),
        # a long prompt chunk on its way into the cache
        dict(a, name="append prompt chunk", n_dec=0, n_chunk=1, chunk=8192, ctx_lo=8192, ctx=8192, Hq=64, Hkv=8),
        # ragged chunks and decode tokens, weights of their own per head, half of each head rotated
        dict(a, name="append ragged", n_dec=11, n_chunk=4, chunk=1501, ctx_lo=50, ctx=2100, Hq=40, Hkv=8, per_head=True,
             rot=64, block_len=128),
        # a shard of 4-bit histories widened for a pass round the ring
        dict(r, name="read 4-bit histories", fmt="fp4", n_seq=8, lo=20000, ctx=65536, Hkv=8),
        # short ragged pieces out of an fp8 cache
        dict(r, name="read fp8 pieces", fmt="fp8", n_seq=23, lo=100, ctx=3001, Hkv=4, block_len=128),
        # decode of a serving batch with ragged histories
        dict(t, name="decode 4-bit", n_dec=64, n_chunk=0, chunk=0, ctx_lo=4096, ctx=16384, Hq=64, Hkv=8),
        # decode over few long histories, wide groups
        dict(t, name="long decode 4-bit", n_dec=8, n_chunk=0, chunk=0, ctx_lo=65536, ctx=131072, Hq=128, Hkv=8, block_len=256),
        # ragged prompt chunks over a 4-bit cache
        dict(t, name="prompts 4-bit", n_dec=0, n_chunk=3, chunk=1501, ctx_lo=1501, ctx=6007, Hq=64, Hkv=8),
        # the smallest call: two short sequences behind one system prompt
        dict(s, name="shared prefix short", n_groups=1, n_seq=2, chunk=1, prefix=512, lo=1, own=64, Hq=8, Hkv=2, d=64),
        # a decoding batch behind one long document
        dict(s, name="shared prefix decode", n_groups=1, n_seq=64, chunk=1, prefix=32768, lo=100, own=1000, Hq=64, Hkv=8),
        # groups of samples of a prompt each, 4-bit pages
        dict(s, name="shared prefix samples 4-bit", fmt="fp4", n_groups=7, n_seq=56, chunk=1, prefix=16384, lo=1, own=3000,
             Hq=128, Hkv=8, block_len=128),
        # questions of some hundred tokens to one document, fp8 pages
        dict(s, name="shared prefix questions fp8", fmt="fp8", n_groups=1, n_seq=16, chunk=301, prefix=16384, lo=301,
             own=900, Hq=64, Hkv=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv, op = rng.choice([1, 2, 4, 8]), rng.choice(["append", "read", "attn", "attn", "shared", "shared"])
    c = dict(op=op, Hkv=Hkv, d=128, block_len=rng.choice([64, 64, 128, 256, 320]))
    if op == "append":
        c.update(fmt="fp4", Hq=Hkv * rng.choice([1, 2, 3, 5, 7, 8, 16]), n_dec=rng.choice([0, 1, _log_int(rng, 2, 200)]),
                 per_head=rng.random() < 0.3, paired=rng.random() < 0.4, rot=rng.choice([16, 64, 128, 128]))
        c.update(n_chunk=0 if c["n_dec"] and rng.random() < 0.4 else rng.randint(1, 4))
        c.update(chunk=_log_int(rng, 2, 4096) if c["n_chunk"] else 0)
        lo = max(1, c["chunk"])
        c.update(ctx_lo=lo, ctx=lo + _log_int(rng, 1, 500))
        return c
    if op == "read":
        c.update(fmt=rng.choice(["fp4", "fp4", "fp8", "bf16"]), n_seq=_log_int(rng, 1, 32), lo=rng.randint(1, 300))
        c.update(ctx=_log_int(rng, 301, 8000))
        if c["fmt"] == "bf16":
            c.update(d=rng.choice([64, 128]))
        return c
    G = rng.choice([1, 2, 4, 8, 8, 16, 3, 5, 6, 7])
    c.update(Hq=Hkv * G)
    if op == "attn":
        kind = rng.choice(["decode", "drafts", "chunk", "mixed"])
        c.update(fmt="fp4", n_dec=0, n_chunk=0, chunk=0)
        if kind == "decode":
            c.update(n_dec=_log_int(rng, 1, 128), ctx_lo=rng.randint(1, 500), ctx=_log_int(rng, 500, 16384))
        elif kind == "drafts":
            c.update(n_chunk=_log_int(rng, 1, 64), chunk=rng.randint(2, 9), ctx_lo=rng.randint(9, 500), ctx=_log_int(rng, 500, 16384))
        elif kind == "chunk":
            c.update(n_chunk=rng.randint(1, 4), chunk=_log_int(rng, 10, 1500))
            c.update(ctx_lo=c["chunk"], ctx=c["chunk"] + _log_int(rng, 1, 8000))
        else:
            c.update(n_dec=_log_int(rng, 1, 40), n_chunk=rng.randint(1, 3), chunk=_log_int(rng, 10, 1500))
            c.update(ctx_lo=c["chunk"], ctx=c["chunk"] + _log_int(rng, 1, 6000))
        w = rng.random() < 0.3
        c.update(window=_log_int(rng, 1, 4096) if w else 0, n_sink=rng.choice([0, 1, 4, 100]) if w else 0)
        return c
    c.update(fmt=rng.choice(["bf16", "bf16", "fp8", "fp4"]), n_groups=rng.choice([1, 1, 1, 2, 3, 9]))
    if c["fmt"] == "bf16":
        c.update(d=rng.choice([64, 128, 128]))
    c.update(chunk=rng.choice([1, 1, rng.randint(2, 9), _log_int(rng, 10, 400)]))
    c.update(n_seq=c["n_groups"] * _log_int(rng, 1, 64 if c["chunk"] < 10 else 8) // rng.choice([1, 1, 2]) + 1)
    c.update(n_seq=min(c["n_seq"], 160, 1 + 4000 // c["chunk"]))
    c.update(prefix=c["block_len"] * max(1, _log_int(rng, 64, 16384) // c["block_len"]), lo=c["chunk"])
    c.update(own=c["lo"] + _log_int(rng, 1, 2000))
    return c


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    r = random.Random(" ".join("%s" % case[k] for k in sorted(case) if k != "name"))
    if case["op"] == "read":
        n = [case["ctx"] if i == 0 else r.randint(case["lo"], max(case["lo"], case["ctx"])) for i in range(case["n_seq"])]
        start = [r.randint(0, 100) if i % 2 else 0 for i in range(len(n))]
        return n, [a + b for a, b in zip(n, start)]
    if case["op"] == "shared":
        q = [case["chunk"] if i == 0 or case["chunk"] < 10 else r.randint(1, case["chunk"]) for i in range(case["n_seq"])]
        own_tokens = [case["own"] if i == 0 else r.randint(max(case["lo"], q[i]), max(case["own"], q[i])) for i in range(len(q))]
        return q, [p + m for p, m in zip(_prefix_of(case), own_tokens)]
    q = [case["chunk"] if i == 0 or case["chunk"] < 10 else r.randint(1, case["chunk"]) for i in range(case["n_chunk"])]
    q += [1] * case["n_dec"]
    s = [case["ctx"] if i == 0 else r.randint(max(case["ctx_lo"], q[i]), max(case["ctx"], q[i])) for i in range(len(q))]
    return q, s


def _groups(case):
    """(first sequence of each group and their number behind them, the groups' prefixes): the first group's
    prefix is the longest."""
    n, k = case["n_seq"], case["n_groups"]
    blocks = case["prefix"] // case["block_len"]
    return [n * i // k for i in range(k + 1)], [max(1, blocks - blocks * i // (2 * k)) * case["block_len"] for i in range(k)]


def _prefix_of(case):
    """The prefix of each sequence."""
    cu, prefix = _groups(case)
    return [p for j, p in enumerate(prefix) for _ in range(cu[j + 1] - cu[j])]


def _reach(case, n, s):
    """(first tokens, first token of the window) that n new tokens of a history of s can see."""
    lo = max(0, s - n - case["window"] + 1) if case.get("window") else 0
    return min(case.get("n_sink", 0), lo), lo


def _token_bytes(case):
    """Bytes of one token's head in the pages."""
    d = case["d"]
    return d // 2 + d // BLOCK if case["fmt"] == "fp4" else d + 4 / SCALE_BLOCK if case["fmt"] == "fp8" else 2 * d


def work(case):
    q, s = _lengths(case)
    T, Hkv, d = sum(q), case["Hkv"], case["d"]
    if case["op"] == "read":
        return {"bytes": 2 * T * Hkv * (_token_bytes(case) + 2 * d), "flops": 2 * T * Hkv * d}
    Hq = case["Hq"]
    if case["op"] == "append":
        tables = 4 * case["rot"] * T  # a row of cosines and one of sines for each token
        return {"bytes": 2 * T * d * (Hq + 2 * Hkv) + 2 * T * d * Hq + 2 * T * Hkv * _token_bytes(case) + tables,
                "flops": T * d * (Hq + Hkv) * 7}
    pairs = tokens = 0
    if case["op"] == "shared":
        cu, prefix = _groups(case)
        tokens = sum(p for j, p in enumerate(prefix) if cu[j + 1] > cu[j])
        for n, m, p in zip(q, s, _prefix_of(case)):
            tokens += m - p
            pairs += n * (m - n) + n * (n + 1) // 2
    else:
        for n, m in zip(q, s):
            w = case["window"] or m
            first, lo = _reach(case, n, m)
            tokens += first + m - lo
            for p in (range(m - n, m) if case["window"] else ()):
                pairs += min(p + 1, w) + min(case["n_sink"], max(0, p + 1 - w))
            if not case["window"]:
                pairs += n * (m - n) + n * (n + 1) // 2
    return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 2 * tokens * Hkv * _token_bytes(case), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ inputs


def _e2m1(x):
    """Codes of x, to the nearest (ties to the even code), +-6 at most."""
    a = x.abs()
    code = (a > 0.25).to(torch.uint8)
    for edge, above in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if above else (a > edge)
    return code | ((x < 0).to(torch.uint8) << 3)


def _quantise4(x, head_scale):
    """4-bit codes, two a byte, and the blocks' scales: x [.., heads, d], head_scale [heads, 1]."""
    blocks = x.unflatten(-1, (-1, BLOCK))
    most = blocks.abs().amax(-1)
    scale = (most / (6.0 * head_scale)).clamp_max(448.0).to(torch.float8_e4m3fn)
    by = (scale.to(x.dtype) * head_scale)[..., None]
    code = _e2m1(torch.where(by > 0, blocks / by, 0.0)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _pairs(dtype):
    """The two values of each byte of codes."""
    table = torch.tensor([[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)], device=DEV)
    return table.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q_lens, seq_lens = _lengths(case)
    T, B, L = sum(q_lens), len(q_lens), case["block_len"]
    Hkv, d, fmt = case["Hkv"], case["d"], case["fmt"]

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    # the pages that a sequence holds: all of its own, or those of its sinks and window
    held = []
    for n, m in zip(q_lens, seq_lens):
        first, lo = _reach(case, n, m)
        held.append([i for i in range(-(-m // L)) if i * L < first or (i + 1) * L > lo])
    n_pages, width = sum(map(len, held)) + 3, max(-(-m // L) for m in seq_lens)
    if case["op"] == "shared":  # a group's first pages are those of its first sequence
        cu, prefix = _groups(case)
        n_pages -= sum(max(0, cu[j + 1] - cu[j] - 1) * (p // L) for j, p in enumerate(prefix))
    shuffled = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    if case["op"] == "shared":
        for j, p in enumerate(prefix):
            if cu[j + 1] > cu[j]:
                table[cu[j] : cu[j + 1], : p // L] = torch.tensor([shuffled.pop() for _ in range(p // L)], dtype=torch.int32)
        held = [blocks[p // L :] for blocks, p in zip(held, _prefix_of(case))]
    for b, blocks in enumerate(held):
        for i in blocks:
            table[b, i] = shuffled.pop()
    s = dict(case=case, block_table=table.to(DEV), seq_lens=torch.tensor(seq_lens, dtype=torch.int32, device=DEV),
             cu_q=torch.tensor([sum(q_lens[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV),
             k_scale=None, v_scale=None, k_head_scale=None, v_head_scale=None)
    if fmt == "fp4":
        # codes and scales of cached tokens: normal values, quantised in pieces
        pages = torch.empty(2, n_pages, Hkv, L, d // 2, dtype=torch.uint8, device=DEV)
        scale = torch.empty(2, n_pages, Hkv, L, d // BLOCK, dtype=torch.float8_e4m3fn, device=DEV)
        heads = torch.rand(2, Hkv, generator=g, device=DEV) * 1.5 + 0.5
        for x in range(2):
            for at in range(0, n_pages, 512):
                n = min(512, n_pages - at)
                codes, by = _quantise4(randn(n, L, Hkv, d, dtype=torch.float32), heads[x][:, None])
                pages[x, at : at + n] = codes.transpose(1, 2)
                scale[x, at : at + n].view(torch.uint8)[:] = by.view(torch.uint8).transpose(1, 2)
        s.update(pages=pages, scale=scale, k_pages=pages[0], v_pages=pages[1], k_scale=scale[0], v_scale=scale[1],
                 k_head_scale=heads[0], v_head_scale=heads[1])
    else:
        for x in "kv":
            p = randn(n_pages, Hkv, L, d)
            if fmt == "fp8":  # e4m3 codes and one scale per (page, head, 64 tokens): amax / 448
                blocks = p.float().view(n_pages, Hkv, L // SCALE_BLOCK, SCALE_BLOCK, d)
                by = blocks.abs().amax((3, 4)).clamp_min(1e-6) / 448.0
                p, s[x + "_scale"] = (blocks / by[..., None, None]).to(torch.float8_e4m3fn).view(n_pages, Hkv, L, d), by
            s[x + "_pages"] = p
    if case["op"] == "read":
        s["n_tokens"] = T
        s["starts"] = torch.tensor([m - n for n, m in zip(q_lens, seq_lens)], dtype=torch.int32, device=DEV)
        return s
    Hq = case["Hq"]
    if case["op"] == "append":
        s["qkv"] = randn(T, (Hq + 2 * Hkv) * d)  # the fused projection's output
        w = (1.0 + 0.2 * torch.randn(Hq + Hkv, d, generator=g, device=DEV)).to(torch.bfloat16)
        s["q_weight"], s["k_weight"] = (w[:Hq], w[Hq:]) if case["per_head"] else (w[0], w[Hq])
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(width * L, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["values"] = _pairs(torch.float32).to(torch.float8_e4m3fn).view(torch.int16).view(-1)  # of each byte, as two e4m3
        return s
    s["q"] = randn(T, Hq, d)
    s["max_q_len"] = max(q_lens)
    if case["op"] == "shared":
        cu, prefix = _groups(case)
        s["cu_groups"], s["prefix_lens"] = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, prefix))
        s["max_group_rows"] = max(sum(q_lens[a:b]) for a, b in zip(cu, cu[1:]))
    # sequences of one chunk length, with the longest history among them (so many that their keys and
    # scores in 32 bits take 16 GB at most)
    s["groups"] = []
    for n in sorted(set(q_lens)):
        rows = [b for b in range(B) if q_lens[b] == n]
        longest = max(seq_lens[b] for b in rows)
        step = max(1, min(64, (1 << 32) // (longest * max(n * Hq, Hkv * d))))
        for i in range(0, len(rows), step):
            some = rows[i : i + step]
            s["groups"].append((n, torch.tensor(some, device=DEV), max(seq_lens[b] for b in some)))
    return s


# ------------------------------------------------------------------ the operators


def run(s):
    return {"append": _append, "read": _read, "attn": _attend, "shared": _attend}[s["case"]["op"]](s)


def _split(s):
    """The queries, keys and values of the fused projection, as views."""
    c = s["case"]
    x = s["qkv"].view(s["qkv"].shape[0], c["Hq"] + 2 * c["Hkv"], c["d"])
    return x[:, : c["Hq"]], x[:, c["Hq"] : c["Hq"] + c["Hkv"]], x[:, c["Hq"] + c["Hkv"] :]


def _append(s):
    """(q, the values of the pages' codes and the blocks' scales, K's and V's)"""
    c = s["case"]
    q, k, v = _split(s)
    if own:
        import mla_decode_attention_gqa_gb300 as skv

        q_out = skv.qk_norm_rope_append(q, k, v, s["k_pages"], s["v_pages"], s["seq_lens"], s["cu_q"], s["block_table"],
                                        cos=s["cos"], sin=s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                        eps=1e-6, interleaved=c["paired"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                        k_head_scale=s["k_head_scale"], v_head_scale=s["v_head_scale"])
        return {"q": q_out, "codes": _values(s), "scales": s["scale"]}
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
    for x, name in ((norm_rope(k, s["k_weight"]), "k"), (v.float(), "v")):
        codes, scale = _quantise4(x, s[name + "_head_scale"][:, None])
        s[name + "_pages"][page, :, at] = codes
        s[name + "_scale"].view(torch.uint8)[page, :, at] = scale.view(torch.uint8)
    return {"q": norm_rope(q, s["q_weight"]).to(q.dtype), "codes": _values(s), "scales": s["scale"]}


def _values(s):
    """What the pages' codes stand for, before their scales (all of them e4m3 values as well)."""
    x = s["values"].index_select(0, s["pages"].view(-1).int())
    return x.view(torch.float8_e4m3fn).view(*s["pages"].shape[:-1], s["case"]["d"])


def _gathered(s, x, page, at):
    """Rows `at` of pages in 32 bits: [.., Hkv, d]."""
    c, pages, scale = s["case"], s[x + "_pages"], s[x + "_scale"]
    if c["fmt"] == "bf16":
        return pages[page, :, at].float()
    if c["fmt"] == "fp8":
        y = pages.view(torch.uint8)[page, :, at].view(pages.dtype).float()
        return y.mul_(scale[page, :, at // SCALE_BLOCK][..., None])
    y = _pairs(torch.float32)[pages[page, :, at].int()].flatten(-2).unflatten(-1, (-1, BLOCK))
    by = scale.view(torch.uint8)[page, :, at].view(scale.dtype).float() * s[x + "_head_scale"][:, None]
    return y.mul_(by[..., None]).flatten(-2)


def _read(s):
    if own:
        import mla_decode_attention_gqa_gb300 as skv

        k, v = skv.kv_read_paged(s["k_pages"], s["v_pages"], s["cu_q"], s["block_table"], n_tokens=s["n_tokens"],
                                 starts=s["starts"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 k_head_scale=s["k_head_scale"], v_head_scale=s["v_head_scale"], scale_block=SCALE_BLOCK)
        return {"k": k, "v": v}
    L = s["case"]["block_len"]
    row = torch.arange(s["n_tokens"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"], row, right=True) - 1
    pos = s["starts"][seq] - s["cu_q"][seq] + row
    page, at = s["block_table"][seq, pos // L].long(), (pos % L).long()
    return {x: _gathered(s, x, page, at).to(torch.bfloat16) for x in "kv"}


def _attend(s):
    c = s["case"]
    if own:
        import mla_decode_attention_gqa_gb300 as skv

        pages = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_head_scale=s["k_head_scale"],
                     v_head_scale=s["v_head_scale"], max_q_len=s["max_q_len"])
        what = (s["q"], s["k_pages"], s["v_pages"], s["seq_lens"], s["cu_q"], s["block_table"])
        if c["op"] == "shared":
            out, lse = skv.attn_shared_prefix_paged(*what, s["cu_groups"], s["prefix_lens"],
                                                    max_group_rows=s["max_group_rows"], **pages)
        else:
            out, lse = skv.attn_chunk_paged(*what, window=c["window"], n_sink=c["n_sink"], **pages)
        return {"out": out, "lse": lse}
    L, Hkv, d, window, n_sink = c["block_len"], c["Hkv"], c["d"], c.get("window", 0), c.get("n_sink", 0)
    G = c["Hq"] // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
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
        k = _gathered(s, "k", page, at)  # [sequences, tokens, Hkv, d]
        p = torch.matmul(q * (1.0 / math.sqrt(d)), k.permute(0, 2, 3, 1))
        p = p.view(len(rows), Hkv, n, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
        top = p.amax(-1, keepdim=True)
        p = p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        v = _gathered(s, "v", page, at)
        o = torch.matmul(p.view(len(rows), Hkv, n * G, -1), v.transpose(1, 2))
        o = o.view(len(rows), Hkv, n, G, d) / total
        out[token] = o.transpose(1, 2).reshape(len(rows), n, c["Hq"], d).to(out.dtype)
        lse[token] = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(len(rows), n, c["Hq"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attend, "shared": _exact_attend}[case["op"]](s)


def _spans(s):
    """(first row, one behind the last, tokens with them) of each sequence."""
    cu, m = s["cu_q"].tolist(), s["seq_lens"].tolist()
    return [(cu[b], cu[b + 1], m[b]) for b in range(len(m))]


def _exact_rows(s, x, page, at):
    """Rows of pages, all heads, from the formats' definitions: [rows, Hkv, d]."""
    c = s["case"]
    y = s[x + "_pages"].view(torch.uint8 if c["fmt"] != "bf16" else torch.bfloat16)[page, :, at]
    if c["fmt"] == "bf16":
        return y.double()
    if c["fmt"] == "fp8":
        y = y.view(torch.float8_e4m3fn).double()
        return y * s[x + "_scale"].double()[page, :, at // SCALE_BLOCK].unsqueeze(-1)
    low, high = y & 15, y >> 4
    code = torch.stack((low, high), -1).flatten(-2).long()
    exponent, mantissa = (code >> 1) & 3, code & 1
    size = torch.where(exponent == 0, mantissa * 0.5, (1 + 0.5 * mantissa.double()) * 2.0 ** (exponent - 1).double())
    value = torch.where(code >= 8, -size, size)
    by = s[x + "_scale"].view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).double()
    return value * by.repeat_interleave(BLOCK, -1) * s[x + "_head_scale"].double()[:, None]


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

    steps = torch.tensor(_E2M1[:8], dtype=torch.float64, device=DEV)
    middle = (steps[1:] + steps[:-1]) / 2
    codes = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)[
        torch.stack((s["pages"] & 15, s["pages"] >> 4), -1).flatten(-2).long()]
    scales = s["scale"].double()
    for n, (x, h) in enumerate(((turned(k, s["k_weight"]), s["k_head_scale"]), (v, s["v_head_scale"]))):
        h = h.double()[:, None]
        x = x.view(*x.shape[:-1], c["d"] // BLOCK, BLOCK)
        by = torch.clamp(x.abs().amax(-1) / (6 * h), max=448.0).to(torch.float8_e4m3fn).double()
        y = x / (by * h).unsqueeze(-1)
        size = y.abs().nan_to_num(0.0)
        # the nearest step; in the middle the one with the even number
        up, down = torch.bucketize(size, middle, right=True), torch.bucketize(size, middle)
        y = torch.copysign(steps[torch.where(up % 2 == 0, up, down)], y).flatten(-2)
        for b, (lo, hi, m) in enumerate(_spans(s)):
            t = torch.arange(m - hi + lo, m, device=DEV)
            page, at = s["block_table"][b].long()[t // L], t % L
            codes[n][page, :, at] = y[lo:hi]
            scales[n][page, :, at] = by[lo:hi]
    return {"q": turned(q, s["q_weight"]), "codes": codes, "scales": scales}


def _exact_read(s):
    L = s["case"]["block_len"]
    found = {"k": [], "v": []}
    for b, (lo, hi, _) in enumerate(_spans(s)):
        t = int(s["starts"][b]) + torch.arange(hi - lo, device=DEV)
        for x in "kv":
            found[x].append(_exact_rows(s, x, s["block_table"][b].long()[t // L], t % L))
    return {x: torch.cat(y) for x, y in found.items()}


def _exact_attend(s):
    c = s["case"]
    G, L, window, n_sink = c["Hq"] // c["Hkv"], c["block_len"], c.get("window", 0), c.get("n_sink", 0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, (lo, hi, m) in enumerate(_spans(s)):
        for r in range(lo, hi, 512):
            e = min(r + 512, hi)
            pos = torch.arange(m - hi + r, m - hi + e, device=DEV)
            start = max(0, m - hi + r - window + 1) if window else 0
            t = torch.arange(start, m - hi + e, device=DEV)
            if start:
                t = torch.cat((torch.arange(min(n_sink, start), device=DEV), t))
            hidden = t[None] > pos[:, None]
            if window:
                hidden |= (pos[:, None] - t[None] >= window) & (t[None] >= n_sink)
            page, at = s["block_table"][b].long()[t // L], t % L
            k, v = _exact_rows(s, "k", page, at), _exact_rows(s, "v", page, at)
            for h in range(c["Hkv"]):
                x = torch.einsum("igd,td->igt", s["q"][r:e, h * G : (h + 1) * G].double(), k[:, h]) / math.sqrt(c["d"])
                x = x.masked_fill(hidden[:, None], -math.inf)
                total = torch.logsumexp(x, -1)
                lse[r:e, h * G : (h + 1) * G] = total
                out[r:e, h * G : (h + 1) * G] = torch.einsum("igt,td->igd", torch.exp(x - total[..., None]), v[:, h])
    return {"out": out, "lse": lse}
