"""4-bit pages past what the attention kernels can address: their block scales are fetched by coordinates of 32 bits
that count two words a token."""

import ctypes

import pytest

import mla_decode_attention_gqa_gb300 as skv
from tests.test_chunk_host import _chunk, _paged
from tests.test_fp4_shared_host import _call_chunk, _call_shared, _fp4, _ref, _shared

MOST = 1 << 30


def _one_page(block_len):
    strides = (4 * 64 * block_len, 64 * block_len, 64)
    return _paged(block_len=block_len, max_blocks=1, num_blocks=1), dict(kv_dtype=2, k_strides=strides, v_strides=strides)


@pytest.mark.parametrize("shared", [False, True])
def test_attention_refuses_pages_that_it_cannot_address(shared):
    lib = skv.load_library()
    for block_len, fits in ((MOST, True), (MOST + 64, False)):
        pg, kw = _one_page(block_len)
        d, n = _chunk(**kw), ctypes.c_size_t(0)
        size = (lib.attn_shared_prefix_paged_workspace_size(_ref(d), _ref(pg), _ref(_shared()), ctypes.byref(n)) if shared
                else lib.attn_chunk_paged_workspace_size(_ref(d), _ref(pg), ctypes.byref(n)))
        assert size == (skv.SKV_OK if fits else skv.SKV_EINVAL)
        # (without a workspace nothing is launched)
        call = _call_shared(d, pg=pg, fp4=_fp4()) if shared else _call_chunk(d, pg=pg)
        assert call == (skv.SKV_EWORKSPACE if fits else skv.SKV_EINVAL)
    pg, kw = _one_page(MOST + 64)
    assert _call_chunk(_chunk(T=0, **kw), pg=pg) == skv.SKV_EINVAL
    for fmt in (0, 1):  # other pages have no such limit
        strides = (4 * 128 * (MOST + 64), 128 * (MOST + 64), 128)
        d = _chunk(kv_dtype=fmt, k_strides=strides, v_strides=strides)
        n = ctypes.c_size_t(0)
        assert lib.attn_chunk_paged_workspace_size(_ref(d), _ref(pg), ctypes.byref(n)) == skv.SKV_OK
