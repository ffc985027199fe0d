"""The first launch of a process, whose warps wait for their instructions one after the other: every head of
qk_norm_rope_append is read before the next copy into its stage."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
import torch
import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged

fmt, T, Hq, Hkv, L = sys.argv[1], 8192, 64, 8, 64
g = torch.Generator(device="cuda").manual_seed(int(sys.argv[2]))
qkv = torch.randn(T, (Hq + 2 * Hkv) * 128, generator=g, device="cuda", dtype=torch.bfloat16)
table = torch.arange(T // L, dtype=torch.int32, device="cuda")[None]
lens = torch.tensor([T], dtype=torch.int32, device="cuda")
cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
cos, sin = paged.rotation_tables(T, 128, device="cuda")
w = torch.ones(128, device="cuda")
kw = {}
if fmt == "fp4":
    k, v, kw["k_scale"], kw["v_scale"] = paged.fp4_pages(T // L, Hkv, L, device="cuda")
elif fmt == "fp8":
    k, v = (torch.zeros(T // L, Hkv, L, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    kw["k_scale"] = kw["v_scale"] = torch.full((T // L, Hkv, 1), 0.02, device="cuda")
else:
    k, v = (torch.zeros(T // L, Hkv, L, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
out = torch.full((T, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
q, kk, vv = paged.split_qkv(qkv, Hq, Hkv)
torch.cuda.synchronize()
skv.qk_norm_rope_append(q, kk, vv, k, v, lens, cu, table, cos=cos, sin=sin, q_weight=w, k_weight=w, q_out=out, **kw)
torch.cuda.synchronize()
x = q.float()
x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
c, s = cos[:, None], sin[:, None]
x = torch.cat((x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s), -1)
# the output's rounding, and 32-bit norm and rotation of a head whose values are below 2^3
bad = ~((out.float() - x).abs() <= 2.0 ** -8 * x.abs() + 2.0 ** -16)
assert skv.device_error() == 0 and not bad.any(), bad.any(-1).nonzero()[:8].tolist()
"""


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_first_launch(fmt):
    for seed in range(2):
        r = subprocess.run([sys.executable, "-c", SCRIPT, fmt, str(seed)], cwd=ROOT, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-2000:]
