"""What the calls over 4-bit pages, kv_read_paged and attn_shared_prefix_paged refuse, on the host and before
any launch, through the C ABI and the binding."""

import ctypes

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged
from tests.test_chunk_host import FAKE, _append, _chunk, _paged, _set

FP4 = dict(kv_dtype=2, k_strides=(4 * 64 * 64, 64 * 64, 64), v_strides=(4 * 64 * 64, 64 * 64, 64))
FP4_APPEND = dict(kv_dtype=2, k_page_strides=FP4["k_strides"], v_page_strides=FP4["v_strides"])


def _fp4(**kw):
    f = skv.SkvFp4Scales(0x10000, 0x10000, None, None)
    for k, v in kw.items():
        setattr(f, k, v)
    return f


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _call_chunk(d, pg=None, fp4="there", ws=None, ws_bytes=0, **ptr):
    lib = skv.load_library()
    p = dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, seq=FAKE, out=FAKE, lse=FAKE)
    p.update(ptr)
    return lib.attn_chunk_paged_fp4(_ref(d), _ref(pg or _paged()), _ref(_fp4() if fp4 == "there" else fp4), p["q"], p["k"],
                                    p["v"], p["cu"], p["seq"], p["out"], p["lse"], ws, ws_bytes, None)


def _call_append(d, pg=None, fp4="there", **ptr):
    lib = skv.load_library()
    p = dict(q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, cos=FAKE, sin=FAKE, pos=None, cu=FAKE, seq=FAKE, out=FAKE, kp=FAKE, vp=FAKE)
    p.update(ptr)
    return lib.qk_norm_rope_append_fp4(_ref(d), _ref(pg or _paged()), _ref(_fp4() if fp4 == "there" else fp4), p["q"], p["k"],
                                       p["v"], p["qw"], p["kw"], p["cos"], p["sin"], p["pos"], p["cu"], p["seq"], p["out"],
                                       p["kp"], p["vp"], None)


def _read(**kw):
    d = skv.SkvReadDesc()
    base = dict(B=3, T=10, Hkv=4, d=128, kv_dtype=2, scale_block=64, k_page_strides=FP4["k_strides"],
                v_page_strides=FP4["v_strides"], k_out_strides=(4 * 128, 128), v_out_strides=(4 * 128, 128))
    return _set(_set(d, base), kw)


def _call_read(d, pg=None, fp4="there", **ptr):
    lib = skv.load_library()
    p = dict(k=FAKE, v=FAKE, ks=None, vs=None, cu=FAKE, st=None, ko=FAKE, vo=FAKE)
    p.update(ptr)
    return lib.kv_read_paged(_ref(d), _ref(pg or _paged()), _ref(_fp4() if fp4 == "there" else fp4), p["k"], p["v"], p["ks"],
                             p["vs"], p["cu"], p["st"], p["ko"], p["vo"], None)


def _shared(**kw):
    s = skv.SkvSharedDesc(2, 0, 0x10000, 0x10000)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call_shared(d, pg=None, shared="there", fp4=None, ws=None, ws_bytes=0, **ptr):
    lib = skv.load_library()
    p = dict(q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, cu=FAKE, seq=FAKE, out=FAKE, lse=FAKE)
    p.update(ptr)
    return lib.attn_shared_prefix_paged(_ref(d), _ref(pg or _paged()), _ref(_shared() if shared == "there" else shared),
                                        _ref(fp4), p["q"], p["k"], p["v"], p["ks"], p["vs"], p["cu"], p["seq"], p["out"],
                                        p["lse"], ws, ws_bytes, None)


PAGES = [
    (dict(kv_dtype=0), skv.SKV_EINVAL),
    (dict(kv_dtype=1), skv.SKV_EINVAL),
    (dict(kv_dtype=3), skv.SKV_EINVAL),
    (dict(d=64), skv.SKV_EUNSUPPORTED),
    (dict(d=96), skv.SKV_EUNSUPPORTED),
    (dict(B=0), skv.SKV_EINVAL),
    (dict(T=-1), skv.SKV_EINVAL),
]


@pytest.mark.parametrize("kw,code", PAGES + [
    (dict(k_strides=(4 * 64 * 64, 64 * 64, 56)), skv.SKV_EINVAL),
    (dict(k_strides=(4 * 64 * 64, 64 * 64, 48)), skv.SKV_EINVAL),
    (dict(v_strides=(4 * 64 * 64, 0, 64)), skv.SKV_EINVAL),
    (dict(window=-1), skv.SKV_EINVAL),
    (dict(n_sink=3), skv.SKV_EINVAL),
    (dict(softmax_scale=-1.0), skv.SKV_EINVAL),
])
def test_chunk_fp4_refuses(kw, code):
    assert _call_chunk(_set(_chunk(**FP4), kw)) == code
    assert skv.last_error()


def test_chunk_fp4_pointers_and_workspace():
    d = _chunk(**FP4)
    for fp4 in (None, _fp4(k_block=None), _fp4(v_block=None), _fp4(k_block=0x10008), _fp4(k_head=0x10002), _fp4(v_head=0x10001)):
        assert _call_chunk(d, fp4=fp4) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "cu", "seq", "out", "lse"):
        assert _call_chunk(d, **{name: None}) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "out"):
        assert _call_chunk(d, **{name: ctypes.c_void_p(0x10008)}) == skv.SKV_EINVAL
    assert _call_chunk(d) == skv.SKV_EWORKSPACE
    n = ctypes.c_size_t(0)
    assert skv.load_library().attn_chunk_paged_workspace_size(_ref(d), _ref(_paged()), ctypes.byref(n)) == skv.SKV_OK
    assert n.value > 0
    assert _call_chunk(d, ws=FAKE, ws_bytes=n.value - 1) == skv.SKV_EWORKSPACE
    assert _call_chunk(d, pg=_paged(block_len=32)) == skv.SKV_EINVAL
    assert _call_chunk(_set(_chunk(**FP4), dict(T=0)), q=None, fp4=None) == skv.SKV_OK


def test_fp4_dtype_is_refused_elsewhere():
    """The calls without 4-bit scales know no such pages."""
    lib = skv.load_library()
    d = _chunk(**FP4)
    assert lib.attn_chunk_paged(_ref(d), _ref(_paged()), *[FAKE] * 3, None, None, *[FAKE] * 4, None, 0, None) == skv.SKV_EINVAL
    a = _append(**FP4_APPEND)
    assert lib.qk_norm_rope_append(_ref(a), _ref(_paged()), *[FAKE] * 7, None, FAKE, FAKE, None, None, *[FAKE] * 3, None) == skv.SKV_EINVAL
    e = skv.SkvDesc()
    e.B = e.Tq = e.Hq = e.Hkv = 1
    e.dk = e.dv = 128
    e.S_max, e.softmax_scale, e.kv_dtype, e.scale_block = 64, 1.0, 2, 64
    n = ctypes.c_size_t(0)
    assert lib.attn_partial_workspace_size(ctypes.byref(e), 1, ctypes.byref(n)) == skv.SKV_EINVAL


@pytest.mark.parametrize("kw,code", PAGES + [
    (dict(k_page_strides=(4 * 64 * 64, 64 * 64, 56)), skv.SKV_EINVAL),
    (dict(rot=8), skv.SKV_EINVAL),
    (dict(eps=-1.0), skv.SKV_EINVAL),
    (dict(q_out_strides=(16 * 128, 100)), skv.SKV_EINVAL),
])
def test_append_fp4_refuses(kw, code):
    assert _call_append(_set(_append(**FP4_APPEND), kw)) == code


def test_append_fp4_pointers():
    d = _append(**FP4_APPEND)
    for fp4 in (None, _fp4(k_block=None), _fp4(v_block=0x10004), _fp4(v_head=0x10001)):
        assert _call_append(d, fp4=fp4) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "cu", "seq", "out", "kp", "vp", "cos"):
        assert _call_append(d, **{name: None}) == skv.SKV_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(kv_dtype=4), skv.SKV_EINVAL),
    (dict(d=64), skv.SKV_EUNSUPPORTED),
    (dict(B=0), skv.SKV_EINVAL),
    (dict(Hkv=0), skv.SKV_EINVAL),
    (dict(T=-1), skv.SKV_EINVAL),
    (dict(k_out_strides=(4 * 128, 100)), skv.SKV_EINVAL),
    (dict(k_out_strides=(4 * 128, 64)), skv.SKV_EINVAL),
    (dict(v_out_strides=(128, 128)), skv.SKV_EINVAL),
    (dict(v_out_strides=(-512, 128)), skv.SKV_EINVAL),
    (dict(v_out_strides=(0, 128)), skv.SKV_EINVAL),
    (dict(k_page_strides=(4 * 64 * 64, 64 * 64, 32)), skv.SKV_EINVAL),
])
def test_read_refuses(kw, code):
    assert _call_read(_read(**kw)) == code


def test_read_pointers():
    d = _read()
    for name in ("k", "v", "cu", "ko", "vo"):
        assert _call_read(d, **{name: None}) == skv.SKV_EINVAL
    for name in ("ko", "vo"):
        assert _call_read(d, **{name: ctypes.c_void_p(0x10008)}) == skv.SKV_EINVAL
    assert _call_read(d, st=ctypes.c_void_p(0x10002)) == skv.SKV_EINVAL
    assert _call_read(d, fp4=None) == skv.SKV_EINVAL
    full = dict(k_page_strides=(4 * 64 * 128, 64 * 128, 128), v_page_strides=(4 * 64 * 128, 64 * 128, 128))
    assert _call_read(_read(kv_dtype=1, **full), fp4=None) == skv.SKV_EINVAL  # no scales
    assert _call_read(_read(kv_dtype=0, **full)) == skv.SKV_EINVAL            # scales of other pages
    assert _call_read(_set(_read(), dict(T=0)), ko=None) == skv.SKV_OK


@pytest.mark.parametrize("kw,sh,code", [
    (dict(window=64), {}, skv.SKV_EINVAL),
    (dict(n_sink=1), {}, skv.SKV_EINVAL),
    ({}, dict(n_groups=0), skv.SKV_EINVAL),
    ({}, dict(n_groups=-1), skv.SKV_EINVAL),
    ({}, dict(cu_groups=None), skv.SKV_EINVAL),
    ({}, dict(prefix_lens=None), skv.SKV_EINVAL),
    ({}, dict(cu_groups=0x10002), skv.SKV_EINVAL),
    (dict(softmax_scale=-2.0), {}, skv.SKV_EINVAL),
    (dict(kv_dtype=2), {}, skv.SKV_EINVAL),
    (dict(kv_dtype=1), {}, skv.SKV_EINVAL),
    (dict(d=96), {}, skv.SKV_EUNSUPPORTED),
    (dict(T=2 ** 30, Hq=64), {}, skv.SKV_EINVAL),
    ({}, {}, skv.SKV_EWORKSPACE),
])
def test_shared_refuses(kw, sh, code):
    assert _call_shared(_chunk(**kw), shared=_shared(**sh)) == code
    assert skv.last_error()


def test_shared_workspace():
    lib = skv.load_library()
    n = ctypes.c_size_t(0)
    assert _call_shared(_chunk(), shared=None) == skv.SKV_EINVAL
    assert _call_shared(_chunk(), fp4=_fp4()) == skv.SKV_EINVAL
    assert lib.attn_shared_prefix_paged_workspace_size(_ref(_chunk()), _ref(_paged()), _ref(_shared()), None) == skv.SKV_EINVAL
    assert lib.attn_shared_prefix_paged_workspace_size(_ref(_chunk()), _ref(_paged()), _ref(_shared()), ctypes.byref(n)) == skv.SKV_OK
    assert _call_shared(_chunk(), ws=FAKE, ws_bytes=n.value - 1) == skv.SKV_EWORKSPACE
    assert _call_shared(_chunk(), ws=ctypes.c_void_p(0x10010), ws_bytes=n.value) == skv.SKV_EWORKSPACE
    assert lib.attn_shared_prefix_paged_workspace_size(_ref(_set(_chunk(), dict(T=0))), _ref(_paged()), _ref(_shared()),
                                                       ctypes.byref(n)) == skv.SKV_OK and n.value == 0
    assert _call_shared(_set(_chunk(), dict(T=0)), q=None) == skv.SKV_OK


def test_binding_refuses_cpu_tensors_and_mixed_arguments():
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    pages = torch.zeros(1, 1, 64, 64, dtype=torch.uint8)
    ints = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: skv.attn_shared_prefix_paged(q, pages, pages, ints[:1], ints, table, ints, ints[:1]),
                 lambda: skv.kv_read_paged(pages, pages, ints, table, n_tokens=1),
                 lambda: skv.attn_chunk_paged(q, pages, pages, ints[:1], ints, table)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    qkv = torch.zeros(1, 4 * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="go together"):
        paged.chunk_step(qkv, 2, 1, pages, pages, ints[:1], ints, table, cu_groups=ints)
    with pytest.raises(ValueError, match="window"):
        paged.chunk_step(qkv, 2, 1, pages, pages, ints[:1], ints, table, cu_groups=ints, prefix_lens=ints[:1], window=5)


def test_fp4_pages_are_empty_and_shaped():
    k, v, ks, vs = paged.fp4_pages(3, 2, 128)
    assert k.shape == v.shape == (3, 2, 128, 64) and k.dtype == torch.uint8
    assert ks.shape == vs.shape == (3, 2, 128, 8) and ks.dtype == torch.float8_e4m3fn
    assert not k.any() and not ks.view(torch.uint8).any()
