"""Plain 64-bit definitions of 4-bit pages (e2m1 codes, e4m3 block scales, fp32 head scales), on the CPU."""

import torch

from tests import chunk_ref as R

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
VALUES = torch.cat((E2M1, -E2M1))
BLOCK = 16


def values_of(codes):
    """The values of packed codes [.., n] -> [.., 2 n]."""
    c = codes.cpu().view(torch.uint8).long()
    return VALUES[torch.stack((c & 15, c >> 4), -1).flatten(-2)]


def scales_of(block):
    return block.cpu().view(torch.uint8).view(torch.float8_e4m3fn).double()


def dense(codes, block, head):
    """Pages [n, Hkv, L, d] in 64 bits."""
    x = values_of(codes) * scales_of(block).repeat_interleave(BLOCK, -1)
    return x if head is None else x * head.cpu().double()[:, None, None]


def random_pages(n, Hkv, L, d, gen, device):
    """Codes of all kinds and scales of sizes as normal values have them, some of them negative or zero."""
    codes = torch.randint(0, 256, (n, Hkv, L, d // 2), generator=gen, dtype=torch.uint8)
    scale = (0.05 + 0.5 * torch.rand(n, Hkv, L, d // BLOCK, generator=gen)) * (1 - 2 * (torch.rand(
        n, Hkv, L, d // BLOCK, generator=gen) < 0.1).float())
    scale[torch.rand(scale.shape, generator=gen) < 0.02] = 0.0
    return codes.to(device), scale.to(torch.float8_e4m3fn).to(device)


def to_fp4(c, head=True, seed=9):
    """A case of chunk_ref.make_case with 4-bit pages; c["dense"]: the same with its pages in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    n, Hkv, L, d = c["k_pages"].shape
    dev = c["q"].device
    out = dict(c)
    for x in "kv":
        out[x + "_pages"], out[x + "_scale"] = random_pages(n, Hkv, L, d, g, dev)
        out[x + "_head_scale"] = (0.5 + torch.rand(Hkv, generator=g)).to(dev) if head else None
    return with_dense(out)


def with_dense(c):
    c["dense"] = dict(c, k_scale=None, v_scale=None, **{
        x + "_pages": dense(c[x + "_pages"], c[x + "_scale"], c[x + "_head_scale"]) for x in "kv"})
    return c


def pages_of(c):
    """The keyword arguments of a call over c's pages."""
    return {x: c[x] for x in ("k_scale", "v_scale", "k_head_scale", "v_head_scale") if c.get(x) is not None}


def make_case(fmt, q_lens, seq_lens, Hq, Hkv, d, **kw):
    """chunk_ref.make_case with pages of a format; c["dense"] is what the definition reads."""
    c = R.make_case(q_lens, seq_lens, Hq, Hkv, d, fp8=fmt == "fp8", **kw)
    if fmt == "fp4":
        return to_fp4(c)
    c["dense"] = c
    return c
