"""One attention layer's step of a server over a paged KV cache.

``chunk_step`` takes the fused projection's output of a packed batch (prompt chunks, proposed
tokens and single decode tokens side by side) and runs the layer's attention: norms and
rotation of the new queries and keys and the write of keys and values into their pages
(``qk_norm_rope_append``), then the attention of every new token over its sequence's pages
(``attn_chunk_paged``).  Nothing is copied to the host and no length is read there, so a step
can be captured into a CUDA graph and replayed after the arrays of lengths were rewritten.
"""

import torch

from . import attn_chunk_paged, qk_norm_rope_append


def split_qkv(qkv, Hq, Hkv):
    """The query, key and value heads [T,H,d] of a fused projection [T, (Hq + 2 Hkv) d], as views."""
    T, width = qkv.shape
    n = Hq + 2 * Hkv
    if width % n:
        raise ValueError(f"the projection's width {width} is not a multiple of its {n} heads")
    x = qkv.view(T, n, width // n)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def rotation_tables(max_pos, rot, base=10000.0, device=None):
    """cos and sin fp32 [max_pos, rot/2] of the angles p * base^(-2j/rot), computed in 64 bits
    (at position 10^6 a 32-bit angle is off by up to 2^-5)."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def chunk_step(qkv, Hq, Hkv, k_pages, v_pages, seq_lens, cu_q, block_table, *, cos=None, sin=None, q_weight=None,
               k_weight=None, eps=1e-6, positions=None, interleaved=False, max_q_len=None, window=0, n_sink=0,
               k_scale=None, v_scale=None, softmax_scale=None, scale_block=64, out=None, lse=None):
    """Append the packed new tokens to the pages and attend: returns (out bf16 [T,Hq,d], lse
    fp32 [T,Hq]).  seq_lens counts the new tokens; the arguments are those of
    qk_norm_rope_append and attn_chunk_paged (max_q_len = 1 for a decode step: without it the
    attention takes a kernel for long chunks)."""
    q, k, v = split_qkv(qkv, Hq, Hkv)
    q = qk_norm_rope_append(q, k, v, k_pages, v_pages, seq_lens, cu_q, block_table, cos=cos, sin=sin,
                            q_weight=q_weight, k_weight=k_weight, eps=eps, positions=positions,
                            interleaved=interleaved, k_scale=k_scale, v_scale=v_scale, scale_block=scale_block)
    return attn_chunk_paged(q, k_pages, v_pages, seq_lens, cu_q, block_table, max_q_len=max_q_len, window=window,
                            n_sink=n_sink, k_scale=k_scale, v_scale=v_scale, softmax_scale=softmax_scale,
                            scale_block=scale_block, out=out, lse=lse)
